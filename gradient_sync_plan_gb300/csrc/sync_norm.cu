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
// set.
#include <algorithm>
#include <climits>

#include "norm_device.cuh"
#include "optim_internal.h"

namespace ddpk {

template <int MEMBERS, int PTRS>
struct SyncTab {
    static constexpr int kMembers = MEMBERS, kPtrs = PTRS;
    int32_t n;
    int32_t tiles;
    int32_t world;
    int32_t div_mode;
    float div_operand;
    int64_t numel[MEMBERS];
    int64_t offset[MEMBERS];     // bucket position of element 0
    int64_t clen[MEMBERS];       // chunk length of the member's bucket
    float inv_clen[MEMBERS];
    int32_t tile_end[MEMBERS];   // inclusive prefix of tiles
    int8_t lead[MEMBERS];        // elements past a 16-byte boundary, at every rank; -1: ranks differ
    char* ptr[PTRS];             // ptr[m * world + r]
};
using SyncSmall = SyncTab<32, 256>;
using SyncLarge = SyncTab<336, 2624>;
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
__device__ __forceinline__ double square(float f) { return (double)f * (double)f; }
__device__ __forceinline__ double square(uint16_t h) { return square(bf16_to_f32(h)); }

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

// E: element type; G: ranks whose loads are in flight together; U: vectors a
// thread takes of a tile, one after the other: with few ranks the registers
// that leaves free hold more blocks per SM, and those the loads in flight.
template <class E, int G, int U, class TAB>
__global__ void __launch_bounds__(kThreads, 4) k_sync_norm(const __grid_constant__ TAB b, double* partials) {
    using V = typename E::V;
    using S = typename E::S;
    constexpr int L = E::L;
    constexpr int kTile = kThreads * U * L;
    __shared__ double sh[kThreads / 32];
    pdl_release();
    pdl_acquire();
    const int world = b.world;
    for (int tile = blockIdx.x; tile < b.tiles; tile += gridDim.x) {
        int lo = 0, hi = b.n - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (b.tile_end[mid] > tile) hi = mid; else lo = mid + 1;
        }
        const int i = lo;
        // pieces: vectors at 16-byte boundaries, or elements where the ranks'
        // pointers do not line up; positions count from e0, [head, tail) are the member's
        const int step = b.lead[i] >= 0 ? L : 1;
        const int64_t e0 = (int64_t)(tile - (i ? b.tile_end[i - 1] : 0)) * kTile - max((int)b.lead[i], 0);
        const int head = e0 < 0 ? (int)-e0 : 0;
        const int tail = (int)min((int64_t)kTile, b.numel[i] - e0);
        const int64_t q0 = b.offset[i] + e0;
        const int j0 = chunk_of(q0 + head, b.clen[i], b.inv_clen[i]);
        const int near = (int)min((int64_t)kTile, (int64_t)(j0 + 1) * b.clen[i] - q0);     // where chunk j0 ends
        char* const* pp = b.ptr + (size_t)i * world;
        auto at = [&](int r) -> const char* { return pp[r]; };
        auto start_of = [&](int j) { return j + 1 == world ? 0 : j + 1; };
        float s = 0.f;
#pragma unroll 1
        for (int a = threadIdx.x * step; a < kTile; a += kThreads * step) {
            const int first = max(a, head), end = min(a + step, tail);
            if (first >= end) continue;
            int j = j0;
            bool whole = end - first == L;
            if (whole && end > near) {
                j = chunk_of(q0 + first, b.clen[i], b.inv_clen[i]);
                whole = q0 + end <= (int64_t)(j + 1) * b.clen[i];
            }
            if (whole) {
                const int64_t byte = (e0 + first) * (int64_t)sizeof(S);
                const V y = average_v<E>(fold_ring_vec<E, G>(at, world, start_of(j), byte), b.div_mode, b.div_operand);
                for (int r = 0; r < world; ++r) st_stream<V>(pp[r] + byte, y);
                s += sum_squares(y);
                continue;
            }
#pragma unroll 1
            for (int e = first; e < end; ++e) {
                j = chunk_of(q0 + e, b.clen[i], b.inv_clen[i]);
                const S y = average_s<E>(fold_ring_scalar<E>(at, world, start_of(j), e0 + e), b.div_mode, b.div_operand);
                for (int r = 0; r < world; ++r) reinterpret_cast<S*>(pp[r])[e0 + e] = y;
                s += sum_squares(y);
            }
        }
        double w = warp_sum(s);
        if (!in_square_range((float)w)) {        // squared again in binary64, from what this thread wrote to rank 0
            const S* mine = reinterpret_cast<const S*>(pp[0]) + e0;
            double d = 0.0;
#pragma unroll 1
            for (int a = threadIdx.x * step; a < kTile; a += kThreads * step)
                for (int e = max(a, head); e < min(a + step, tail); ++e) d += square(mine[e]);
            w = warp_sum(d);
        }
        const double t = block_sum(w, sh);
        if (threadIdx.x == 0) partials[tile] = t;
        __syncthreads();                         // sh is free for the next tile
    }
}

// Vectors a thread takes of a tile: enough loads in flight with few ranks.
static int vecs_of(int world) { return world <= 2 ? 4 : world <= 4 ? 2 : 1; }

int64_t sync_norm_tile(int world, int dtype) { return (int64_t)kThreads * vecs_of(world) * (dtype == DDP_BF16 ? 8 : 4); }

// Elements past a 16-byte boundary that every rank's pointer is, or -1.
static int lead_of(int world, const SyncMember& m, int64_t es) {
    const uintptr_t q = reinterpret_cast<uintptr_t>(m.ptrs[0]) % 16;
    for (int r = 1; r < world; ++r)
        if (reinterpret_cast<uintptr_t>(m.ptrs[r]) % 16 != q) return -1;
    return (int)((int64_t)q / es);
}

template <class E, int G, int U, class TAB>
static cudaError_t sync_tables(int world, const SyncMember* members, int64_t n, DivSpec div, double* partials,
                               cudaStream_t st) {
    constexpr int64_t kTile = (int64_t)kThreads * U * E::L;
    const int most = std::min(TAB::kMembers, TAB::kPtrs / world);
    TAB b;
    b.world = world;
    b.div_mode = div.mode;
    b.div_operand = div.operand;
    int64_t i = 0;
    while (i < n) {
        b.n = 0;
        b.tiles = 0;
        for (; i < n && b.n < most; ++i, ++b.n) {
            const SyncMember& m = members[i];
            const int lead = lead_of(world, m, (int64_t)sizeof(typename E::S));
            b.tiles += (int32_t)((std::max(lead, 0) + m.numel + kTile - 1) / kTile);
            b.numel[b.n] = m.numel;
            b.offset[b.n] = m.offset;
            b.clen[b.n] = m.clen;
            b.inv_clen[b.n] = 1.0f / (float)m.clen;
            b.tile_end[b.n] = b.tiles;
            b.lead[b.n] = (int8_t)lead;
            for (int r = 0; r < world; ++r) b.ptr[(size_t)b.n * world + r] = static_cast<char*>(m.ptrs[r]);
        }
        const cudaError_t e = launch_dependent(k_sync_norm<E, G, U, TAB>, dim3(cap_ctas(b.tiles)), dim3(kThreads), 0, st,
                                               b, partials);
        if (e != cudaSuccess) return e;
        partials += b.tiles;
    }
    return cudaSuccess;
}

template <class E, class TAB>
static cudaError_t sync_world(int world, const SyncMember* m, int64_t n, DivSpec div, double* partials, cudaStream_t st) {
    if (world <= 2) return sync_tables<E, 2, 4, TAB>(world, m, n, div, partials, st);
    if (world <= 4) return sync_tables<E, 4, 2, TAB>(world, m, n, div, partials, st);
    return sync_tables<E, 8, 1, TAB>(world, m, n, div, partials, st);
}

template <class E>
static cudaError_t sync_size(int world, const SyncMember* m, int64_t n, DivSpec div, double* partials, cudaStream_t st) {
    if (n <= SyncSmall::kMembers && n * world <= SyncSmall::kPtrs)
        return sync_world<E, SyncSmall>(world, m, n, div, partials, st);
    return sync_world<E, SyncLarge>(world, m, n, div, partials, st);
}

cudaError_t launch_sync_norm(int world, const SyncMember* members, int64_t n, int dtype, DivSpec div, double* partials,
                             cudaStream_t st) {
    if (dtype == DDP_F32) return sync_size<EF32>(world, members, n, div, partials, st);
    if (dtype == kDtypeHook) return sync_size<EHOOK>(world, members, n, div, partials, st);
    if (dtype == kDtypeHook16) return sync_size<EHOOK16>(world, members, n, div, partials, st);
    return sync_size<EBF16>(world, members, n, div, partials, st);
}

int64_t sync_norm_tiles(int world, const SyncMember& m, int dtype) {
    const int64_t t = sync_norm_tile(world, dtype);
    return (std::max(lead_of(world, m, elem_bytes(dtype)), 0) + m.numel + t - 1) / t;
}

}  // namespace ddpk
