// sync_norm.cu -- the view sync of a whole step with the gradients' norm in
// its epilogue.
//
// The sync is the fused view of bucket_kernels.cu ("DDP 与 Ring All-Reduce：梯度
// 同步不是一次 AllReduce 就完事", section 05): each element is read from every
// rank, folded in the ring order of the chunk its bucket position falls in,
// divided and written back to every rank.  The value that is written is in a
// register, so its square costs no memory traffic: the norm's own pass over
// one rank's gradients, S of the sync's 2 N S bytes, goes away.
//
// HBM bounds it.  A tile is one block's worth of 16-byte vectors at aligned
// addresses of one member; a member whose pointers share their offset from a
// 16-byte boundary at every rank is cut there, so packed buckets with odd
// member sizes stay on vectors.  A thread places its vector by its bucket
// position; the vectors that a member's end or a chunk boundary cuts go element
// by element.  Blocks take tiles in address order, one each unless a CTA cap is
// set.  355M fp32 on 8 ranks: 3.23 ms, 7.02 TB/s; the sync without a norm takes
// 3.20, a norm pass after it 0.20 more.
#include <algorithm>
#include <climits>

#include "norm_device.cuh"
#include "optim_internal.h"

namespace ddpk {

constexpr uint32_t kRanksDiffer = 15;

struct Member {                  // side by side: a block finds one line of a cold constant cache, not one a field
    int64_t numel;
    int64_t offset;              // bucket position of element 0
    int64_t clen;                // chunk length of the member's bucket
    float inv_clen;
    uint32_t first : 28;         // its first tile
    uint32_t lead : 4;           // elements past a 16-byte boundary, at every rank; kRanksDiffer
};
static_assert(sizeof(Member) == kSyncEntry, "the workspace counts on it");

struct SyncHead {
    int32_t n;
    int32_t tiles;
    int32_t world;
    int32_t vecs;                // vectors a thread takes of a tile
    int32_t div_mode;
    float div_operand;
};
template <int MEMBERS, int PTRS>
struct SyncTab : SyncHead {
    static constexpr bool kDevice = false;
    static constexpr int kMembers = MEMBERS, kPtrs = PTRS;
    int32_t tile_end[MEMBERS];   // inclusive prefix of tiles
    Member member[MEMBERS];
    char* ptr[PTRS];             // ptr[m * world + r]
};
struct SyncDev : SyncHead {      // the same in device memory
    static constexpr bool kDevice = true;
    const int32_t* tile_end;
    const Member* member;
    char* const* ptr;
};
using SyncSmall = SyncTab<32, 256>;
using SyncMedium = SyncTab<176, 704>;
using SyncLarge = SyncTab<304, 2688>;
static_assert(sizeof(SyncLarge) + 16 <= kMaxParamBytes, "sync table exceeds the kernel parameter limit");

// Ring chunk of bucket position q: the quotient from a binary32 estimate, off
// by at most one (chunks are fewer than 2^10), then put right.
__device__ __forceinline__ int chunk_of(int64_t q, int64_t clen, float inv) {
    int j = (int)((float)q * inv);
    if ((int64_t)j * clen > q) --j;
    else if ((int64_t)(j + 1) * clen <= q) ++j;
    return j;
}

template <class E>
__device__ __forceinline__ typename E::V average_v(typename E::V y, int mode, float op) {
    if (mode == kDivPow2) return E::template vdiv<kDivPow2>(y, op);
    if (mode == kDivIeee) return E::template vdiv<kDivIeee>(y, op);
    return E::template vdiv<kDivNone>(y, op);    // the hooks round a lone rank's value here
}
template <class E>
__device__ __forceinline__ typename E::S average_s(typename E::S y, int mode, float op) {
    if (mode == kDivPow2) return E::template sdiv<kDivPow2>(y, op);
    if (mode == kDivIeee) return E::template sdiv<kDivIeee>(y, op);
    return E::template sdiv<kDivNone>(y, op);
}
__device__ __forceinline__ float f32_of(float f) { return f; }
__device__ __forceinline__ float f32_of(uint16_t h) { return bf16_to_f32(h); }

__device__ __forceinline__ float sum_squares(float4 y) {
    return fmaf(y.x, y.x, y.y * y.y) + fmaf(y.z, y.z, y.w * y.w);
}
__device__ __forceinline__ float sum_squares(uint4 y) {
    float s = 0.f;
#pragma unroll
    for (int l = 0; l < 8; ++l) s = fmaf(f32_of(y, l), f32_of(y, l), s);
    return s;
}
__device__ __forceinline__ float sum_squares(float f) { return f * f; }
__device__ __forceinline__ float sum_squares(uint16_t h) { return sum_squares(bf16_to_f32(h)); }

// Zero if and only if every value is a zero of either sign.
__device__ __forceinline__ uint32_t magnitude_bits(float f) { return __float_as_uint(f) << 1; }
__device__ __forceinline__ uint32_t magnitude_bits(uint16_t h) { return (uint32_t)(h & 0x7FFFu); }
__device__ __forceinline__ uint32_t magnitude_bits(float4 y) {
    return (__float_as_uint(y.x) | __float_as_uint(y.y) | __float_as_uint(y.z) | __float_as_uint(y.w)) << 1;
}
__device__ __forceinline__ uint32_t magnitude_bits(uint4 y) { return (y.x | y.y | y.z | y.w) & 0x7FFF7FFFu; }

// E: element type; G: ranks whose loads are in flight together; B: vectors a
// thread folds side by side; MINB: blocks an SM has room for; FEW: there are few
// tiles, and latency counts: a short one goes an element a thread, where a
// vector's cut ends would go one after the other.
template <class E, int G, int B, int MINB, bool FEW, class TAB>
__global__ void __launch_bounds__(kThreads, MINB) k_sync_norm(const __grid_constant__ TAB b, double* partials,
                                                              const __grid_constant__ NormFinish finish) {
    using V = typename E::V;
    using S = typename E::S;
    constexpr int L = E::L;
    constexpr int kRow = kThreads * L;           // elements the block takes with one vector a thread
    __shared__ SquareScratch scratch;
    __shared__ int slot;
    init_squares(scratch);
    AcquireOnce acquire;
    pdl_release();
    if constexpr (TAB::kDevice) acquire();
    const int world = b.world;
    for (int tile = blockIdx.x; tile < b.tiles; tile += gridDim.x) {
        const int i = block_first_past(b.tile_end, b.n, tile, &slot);
        // positions count from e0, which is at a 16-byte boundary if the ranks'
        // pointers line up; [head, tail) are the member's
        const int tile_len = kRow * b.vecs;
        const int lead = b.member[i].lead != kRanksDiffer ? (int)b.member[i].lead : 0;
        const int64_t e0 = (int64_t)(tile - (int)b.member[i].first) * tile_len - lead;
        const int head = e0 < 0 ? (int)-e0 : 0;
        const int tail = (int)min((int64_t)tile_len, b.member[i].numel - e0);
        // pieces: vectors, or elements where the ranks' pointers do not line up
        const int step = b.member[i].lead != kRanksDiffer && !(FEW && tail - head <= kThreads) ? L : 1;
        const int64_t q0 = b.member[i].offset + e0;
        const int j0 = chunk_of(q0 + head, b.member[i].clen, b.member[i].inv_clen);
        const int near = (int)min((int64_t)tile_len, (int64_t)(j0 + 1) * b.member[i].clen - q0);     // where chunk j0 ends
        char* const* pp = b.ptr + (size_t)i * world;
        auto at = [&](int r) -> const char* { return pp[r]; };
        auto start_of = [&](int j) { return j + 1 == world ? 0 : j + 1; };
        acquire();
        float s = 0.f;
        uint32_t bits = 0;                       // of every value's, but the sign
        int a = 0;
        if (B > 1 && step == L && head == 0) {   // rows of whole vectors of chunk j0, several at a time
#pragma unroll 1
            for (; a + B * kRow <= min(tail, near); a += B * kRow) {
                const int64_t byte = (e0 + a + (int)threadIdx.x * L) * (int64_t)sizeof(S);
                V y[B];
                fold_ring_vecs<E, G, B>(at, world, start_of(j0), byte, kThreads * 16, y);
#pragma unroll
                for (int u = 0; u < B; ++u) y[u] = average_v<E>(y[u], b.div_mode, b.div_operand);
                for (int r = 0; r < world; ++r)
#pragma unroll
                    for (int u = 0; u < B; ++u) st_stream<V>(pp[r] + byte + u * (kThreads * 16), y[u]);
#pragma unroll
                for (int u = 0; u < B; ++u) s += sum_squares(y[u]), bits |= magnitude_bits(y[u]);
            }
        }
#pragma unroll 1
        for (a += threadIdx.x * step; a < tail; a += kThreads * step) {
            const int first = max(a, head), end = min(a + step, tail);
            if (first >= end) continue;
            int j = j0;
            bool whole = end - first == L;
            if (whole && end > near) {
                j = chunk_of(q0 + first, b.member[i].clen, b.member[i].inv_clen);
                whole = q0 + end <= (int64_t)(j + 1) * b.member[i].clen;
            }
            if (whole) {
                const int64_t byte = (e0 + first) * (int64_t)sizeof(S);
                const V y = average_v<E>(fold_ring_vec<E, G>(at, world, start_of(j), byte), b.div_mode, b.div_operand);
                for (int r = 0; r < world; ++r) st_stream<V>(pp[r] + byte, y);
                s += sum_squares(y);
                bits |= magnitude_bits(y);
                continue;
            }
#pragma unroll 1
            for (int e = first; e < end; ++e) {
                j = chunk_of(q0 + e, b.member[i].clen, b.member[i].inv_clen);
                const S y = average_s<E>(fold_ring_scalar<E>(at, world, start_of(j), e0 + e), b.div_mode, b.div_operand);
                for (int r = 0; r < world; ++r) reinterpret_cast<S*>(pp[r])[e0 + e] = y;
                s += sum_squares(y);
                bits |= magnitude_bits(y);
            }
        }
        const double t = block_squares(s, bits != 0, scratch, [&] {          // from what the block wrote to rank 0
            const S* mine = reinterpret_cast<const S*>(pp[0]) + e0;
            WideSquares w[2];
#pragma unroll 1
            for (int e = head + (int)threadIdx.x; e < tail; e += 2 * kThreads) {
                w[0].add(f32_of(mine[e]));
                if (e + kThreads < tail) w[1].add(f32_of(mine[e + kThreads]));
            }
            return total(w[0], w[1]);
        });
        if (threadIdx.x == 0) partials[tile] = t;
        __syncthreads();                         // scratch and slot are free for the next tile
    }
    finish_norms<kThreads>(finish, partials, scratch.d);
}

// Vectors a thread takes of a tile: more of them share a block's fixed costs
// (its start, the search, the sum), fewer spread a small call over the SMs,
// and over many ranks one keeps each rank's stream in address order: 355M fp32
// on 8 ranks 3.23 ms with one, 3.32 with four; on 5 ranks 2.25 and 2.07 ms.
constexpr int kSms = 152;
int sync_norm_vecs(int world, int64_t numel, int dtype) {
    const int64_t vectors = numel / (16 / elem_bytes(dtype));
    int v = world <= 7 ? 4 : 1;
    while (v > 1 && vectors < (int64_t)v * kThreads * kSms * 8) v /= 2;
    return v;
}

// Elements past a 16-byte boundary that every rank's pointer is, or -1.
static int lead_of(int world, const SyncMember& m, int64_t es) {
    const uintptr_t q = reinterpret_cast<uintptr_t>(m.ptrs[0]) % 16;
    for (int r = 1; r < world; ++r)
        if (reinterpret_cast<uintptr_t>(m.ptrs[r]) % 16 != q) return -1;
    return (int)((int64_t)q / es);
}

// Launches to make, each with its table: of the smallest capacity that takes
// them all, since a launch's parameters are copied for every eager launch.
struct SyncPlan {
    int world = 0, dtype = 0;
    int32_t tiles = 0;
    std::vector<SyncSmall> small;
    std::vector<SyncMedium> medium;
    std::vector<SyncLarge> large;
    DeviceTable device;                          // more members than one launch's table takes, for little data
    SyncDev dev{};                               // with offsets for addresses
};

const DeviceTable* sync_plan_table(const SyncPlan& plan) { return plan.device.image.empty() ? nullptr : &plan.device; }

// Members [i, n) as far as `most` goes into one table; returns where it stopped.
template <class Ends, class Entries, class Ptrs>
static int64_t fill_table(const SyncMember* members, int64_t i, int64_t n, int64_t most, int world, int dtype, int vecs,
                          DivSpec div, SyncHead* b, Ends ends, Entries entries, Ptrs ptrs) {
    const int64_t es = elem_bytes(dtype), tile = (int64_t)kThreads * vecs * (16 / es);
    *b = SyncHead{0, 0, world, vecs, div.mode, div.operand};
    for (; i < n && b->n < most; ++i, ++b->n) {
        const SyncMember& m = members[i];
        const int lead = lead_of(world, m, es);
        entries[b->n] = Member{m.numel, m.offset, m.clen, 1.0f / (float)m.clen, (uint32_t)b->tiles,
                               lead < 0 ? kRanksDiffer : (uint32_t)lead};
        b->tiles += (int32_t)((std::max(lead, 0) + m.numel + tile - 1) / tile);
        ends[b->n] = b->tiles;
        for (int r = 0; r < world; ++r) ptrs[(size_t)b->n * world + r] = static_cast<char*>(m.ptrs[r]);
    }
    return i;
}

template <class TAB>
static void fill_tables(SyncPlan* plan, const SyncMember* members, int64_t n, int vecs, DivSpec div,
                        std::vector<TAB>* out) {
    const int most = std::min(TAB::kMembers, TAB::kPtrs / plan->world);
    for (int64_t i = 0; i < n;) {
        out->emplace_back();
        TAB& b = out->back();
        i = fill_table(members, i, n, most, plan->world, plan->dtype, vecs, div, &b, b.tile_end, b.member, b.ptr);
        plan->tiles += b.tiles;
    }
}

static void fill_device(SyncPlan* plan, const SyncMember* members, int64_t n, int vecs, DivSpec div) {
    DeviceTable& t = plan->device;
    t.entries_at = (4 * n + 15) / 16 * 16;
    t.more_at = t.entries_at + n * kSyncEntry;
    t.image.assign((size_t)(t.more_at + (8 * n * plan->world + 15) / 16 * 16), 0);
    fill_table(members, 0, n, n, plan->world, plan->dtype, vecs, div, &plan->dev,
               reinterpret_cast<int32_t*>(t.image.data()), reinterpret_cast<Member*>(t.image.data() + t.entries_at),
               reinterpret_cast<char**>(t.image.data() + t.more_at));
    plan->tiles = plan->dev.tiles;
}

template <class TAB>
static bool fits(int world, int64_t n) { return n <= std::min(TAB::kMembers, TAB::kPtrs / world); }

std::shared_ptr<const SyncPlan> make_sync_plan(int world, const SyncMember* members, int64_t n, int vecs, int dtype,
                                               DivSpec div) {
    auto plan = std::make_shared<SyncPlan>();
    plan->world = world;
    plan->dtype = dtype;
    if (fits<SyncSmall>(world, n)) fill_tables(plan.get(), members, n, vecs, div, &plan->small);
    else if (fits<SyncMedium>(world, n)) fill_tables(plan.get(), members, n, vecs, div, &plan->medium);
    else {
        int64_t bytes = 0;
        for (int64_t i = 0; i < n; ++i) bytes += 2 * members[i].numel * elem_bytes(dtype) * world;
        const int64_t most = std::min(SyncLarge::kMembers, SyncLarge::kPtrs / world);
        if (table_on_device((n + most - 1) / most, bytes)) fill_device(plan.get(), members, n, vecs, div);
        else fill_tables(plan.get(), members, n, vecs, div, &plan->large);
    }
    return plan;
}

// Tiles up to which a launch adds its partials itself: a block that arrives
// waits for its stores first, which costs more than a second launch where there
// are waves of blocks (3M elements on 3 ranks, 3100 tiles: 29 against 26 us).
constexpr int32_t kSyncFinishTiles = 608;

template <class E, int G, int B, int MINB, bool FEW, class TAB>
static cudaError_t sync_tables(const TAB* tables, size_t n, double* partials, const NormFinish& finish, cudaStream_t st) {
    for (size_t k = 0; k < n; ++k) {
        const cudaError_t e = launch_table(k_sync_norm<E, G, B, MINB, FEW, TAB>, dim3(cap_ctas(tables[k].tiles)),
                                           dim3(kThreads), st, tables[k], partials, finish);
        if (e != cudaSuccess) return e;
        partials += tables[k].tiles;
    }
    return cudaSuccess;
}

template <class E, class TAB>
static cudaError_t sync_world(int world, bool few, const TAB* tables, size_t n, double* partials,
                              const NormFinish& finish, cudaStream_t st) {
    // 355M fp32: 6.9 TB/s on 2 and 5 ranks, 6.8 on 3, 7.0 on 4 and 8; without
    // side-by-side vectors 6.2 on 2, with four blocks an SM 6.2 on 3, with four
    // blocks of 8 ranks' loads 6.7 on 8.  The same shapes run the other types:
    // bf16 6.4 TB/s on 2 ranks, 6.9 on 4 and 8; the bf16 hook 6.7, 6.9 and 6.9,
    // the fp16 hook 6.5, 6.9 and 6.9.  Two vectors of 16-bit or hook arithmetic
    // side by side spill 56 to 100 bytes, tables in device memory 52 to 288 but
    // in the shape of eight ranks' loads
    if (world <= 2) return sync_tables<E, 2, 2, 4, false>(tables, n, partials, finish, st);
    // eight ranks' loads at a time: 181 tensors of 2336 elements on 13 ranks 10.0
    // against 15.9 us (no gain on up to 4 ranks)
    if (few && world > 4) return sync_tables<E, 8, 1, 3, true>(tables, n, partials, finish, st);
    return sync_tables<E, 4, 1, 5, false>(tables, n, partials, finish, st);
}

template <class E>
static cudaError_t sync_size(const SyncPlan& p, NormSpace ws, const NormFinish& f, cudaStream_t st) {
    const bool few = p.tiles <= kSyncFinishTiles;
    auto run = [&](const auto& t) { return sync_world<E>(p.world, few, t.data(), t.size(), ws.partials, f, st); };
    if (!p.small.empty()) return run(p.small);
    if (!p.medium.empty()) return run(p.medium);
    if (p.device.image.empty()) return run(p.large);
    SyncDev d = p.dev;
    d.tile_end = reinterpret_cast<const int32_t*>(ws.table);
    d.member = reinterpret_cast<const Member*>(ws.table + p.device.entries_at);
    d.ptr = reinterpret_cast<char* const*>(ws.table + p.device.more_at);
    return sync_world<E>(p.world, few, &d, 1, ws.partials, f, st);
}

cudaError_t launch_sync_norm(const SyncPlan& p, NormSpace ws, float* norms, cudaStream_t st) {
    const int32_t first[2] = {0, p.tiles};
    const size_t launches = p.small.size() + p.medium.size() + p.large.size() + (p.device.image.empty() ? 0 : 1);
    const NormFinish f = norm_finish(ws, first, 1, p.world, norms, launches == 1 && p.tiles <= kSyncFinishTiles);
    cudaError_t e;
    if (p.dtype == DDP_F32) e = sync_size<EF32>(p, ws, f, st);
    else if (p.dtype == kDtypeHook) e = sync_size<EHOOK>(p, ws, f, st);
    else if (p.dtype == kDtypeHook16) e = sync_size<EHOOK16>(p, ws, f, st);
    else e = sync_size<EBF16>(p, ws, f, st);
    if (e != cudaSuccess || f.counter) return e;
    return launch_norm_final(ws.partials, first, 1, p.world, norms, st);
}

}  // namespace ddpk
