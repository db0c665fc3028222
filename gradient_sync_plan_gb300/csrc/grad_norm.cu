// grad_norm.cu -- the global gradient norm over many tensors, and clipping.
//
//   norms[r] = sqrt(sum over rank r's tensors and elements of g^2)
//   g <- c g,  c = min(1, max_norm / (norms[r] + 1e-6)),  rounded once to g's type
//
// Both walk a table of byte ranges (tensors that lie back to back are one),
// cut into tiles at 128-byte boundaries of memory: every 16-byte access is
// aligned wherever a tensor starts, and only a range's first and last vector
// are taken element by element.  The tables are filled once and travel in the
// kernels' parameters.  A norm block takes a run of up to sixteen tiles and
// leaves one partial sum; runs depend on the tensors alone and partials are added in a
// fixed order, so a norm does not depend on the grid that computed it.
#include <cooperative_groups.h>

#include <algorithm>
#include <climits>

#include "norm_device.cuh"
#include "optim_internal.h"

namespace ddpk {

struct Range {                 // side by side: a block finds one line of a cold constant cache, not one a field
    char* ptr;
    int64_t bytes;
    int32_t first;             // its first tile
    int32_t rank;
};
static_assert(sizeof(Range) == kRangeEntry, "the workspace counts on it");

template <int CAP>
struct RangeTab {
    static constexpr bool kDevice = false;
    int32_t n;
    int32_t tiles;             // a multiple of `run`
    int32_t run;               // tiles a norm block takes: never of two ranks
    int32_t tile_end[CAP];     // inclusive prefix of tiles; a rank's last range has the padding to a whole run
    Range range[CAP];
};
struct RangeDev {              // the same in device memory
    static constexpr bool kDevice = true;
    int32_t n, tiles, run;
    const int32_t* tile_end;
    const Range* range;
};
// Capacities: a launch's parameters are copied for every eager launch.
constexpr int kNormVecs = (int)(kNormTile / 16 / kThreads);      // vectors a thread takes of a tile
constexpr int64_t kWarpTile = 32 * kNormVecs * 16;               // bytes of a warp's tile
constexpr int kSmallTiles = 128;                                 // warp tiles a rank that k_norm_small takes
constexpr int kRangesSmall = 32;
constexpr int kRangesMedium = 320;
constexpr int kRangesLarge = 1152;
static_assert(sizeof(RangeTab<kRangesLarge>) + sizeof(NormFinish) + 64 <= kMaxParamBytes,
              "range table exceeds the kernel parameter limit");

struct RangePlan {
    int cap = 0;
    std::vector<RangeTab<kRangesSmall>> small;
    std::vector<RangeTab<kRangesMedium>> medium;
    std::vector<RangeTab<kRangesLarge>> large;
    int32_t run = 1;
    std::vector<int32_t> rank_first;             // first partial of each rank, and their end
    // more ranges than one launch's table takes, for little data
    DeviceTable device;
    RangeDev dev{};                              // with offsets for addresses
    // a few warp tiles a rank: what k_norm_small walks, and each rank's first
    std::vector<RangeTab<kRangesSmall>> tiny_small;
    std::vector<RangeTab<kRangesMedium>> tiny_medium;
    std::vector<int32_t> tiny_first;
};

static int64_t range_tiles(const GradRange& g, int64_t tile) {
    const int64_t lead = (int64_t)(reinterpret_cast<uintptr_t>(g.ptr) % kNormAlign);
    return (lead + g.bytes + tile - 1) / tile;
}

// Fills one table with ranges [i, n) as far as `most` goes; returns where it
// stopped.  `rank` counts the ranks whose first partial is known.
template <class Ends, class Entries>
static int64_t fill_table(const GradRange* ranges, int64_t i, int64_t n, int64_t most, int64_t tile, int run,
                          int64_t partials, int* rank, std::vector<int32_t>* rank_first, Ends ends, Entries entries,
                          int32_t* count, int32_t* all_tiles) {
    int64_t tiles = 0, k = 0;
    for (; i < n && k < most; ++i, ++k) {
        while (*rank < ranges[i].rank) (*rank_first)[++*rank] = (int32_t)(partials + tiles / run);
        const int64_t first = tiles;
        tiles += range_tiles(ranges[i], tile);
        if (k + 1 == most || i + 1 == n || ranges[i + 1].rank != ranges[i].rank) tiles = (tiles + run - 1) / run * run;
        ends[k] = (int32_t)tiles;
        entries[k] = Range{ranges[i].ptr, ranges[i].bytes, (int32_t)first, ranges[i].rank};
    }
    *count = (int32_t)k;
    *all_tiles = (int32_t)tiles;
    return i;
}

template <int CAP>
static void fill_tables(const GradRange* ranges, int64_t n, int ranks, int64_t tile, int run,
                        std::vector<RangeTab<CAP>>* out, std::vector<int32_t>* rank_first) {
    rank_first->assign(ranks + 1, 0);
    int64_t partials = 0;
    int rank = 0;
    for (int64_t i = 0; i < n;) {
        out->emplace_back();
        RangeTab<CAP>& b = out->back();
        b.run = run;
        i = fill_table(ranges, i, n, CAP, tile, run, partials, &rank, rank_first, b.tile_end, b.range, &b.n, &b.tiles);
        partials += b.tiles / run;
    }
    while (rank < ranks) (*rank_first)[++rank] = (int32_t)partials;
}

static void fill_device(const GradRange* ranges, int64_t n, int ranks, RangePlan* plan) {
    DeviceTable& t = plan->device;
    t.entries_at = (4 * n + 15) / 16 * 16;
    t.image.assign((size_t)(t.entries_at + (n * kRangeEntry + 15) / 16 * 16), 0);
    plan->rank_first.assign(ranks + 1, 0);
    int rank = 0;
    plan->dev.run = plan->run;
    fill_table(ranges, 0, n, n, kNormTile, plan->run, 0, &rank, &plan->rank_first,
               reinterpret_cast<int32_t*>(t.image.data()), reinterpret_cast<Range*>(t.image.data() + t.entries_at),
               &plan->dev.n, &plan->dev.tiles);
    while (rank < ranks) plan->rank_first[++rank] = plan->dev.tiles / plan->run;
}

const DeviceTable* range_plan_table(const RangePlan& plan) {
    return plan.device.image.empty() ? nullptr : &plan.device;
}

static RangeDev device_ranges(const RangePlan& plan, const char* table) {
    RangeDev d = plan.dev;
    d.tile_end = reinterpret_cast<const int32_t*>(table);
    d.range = reinterpret_cast<const Range*>(table + plan.device.entries_at);
    return d;
}

std::shared_ptr<const RangePlan> make_range_plan(const GradRange* ranges, int64_t n, int ranks) {
    auto plan = std::make_shared<RangePlan>();
    int64_t tiles = 0;
    std::vector<int64_t> warp_tiles(ranks, 0);
    for (int64_t i = 0; i < n; ++i) {
        tiles += range_tiles(ranges[i], kNormTile);
        warp_tiles[ranges[i].rank] += range_tiles(ranges[i], kWarpTile);
    }
    // One wave of eight blocks an SM while a run of kNormOneWave makes it; then
    // runs of four, whose blocks the SMs take as they get free.
    const int64_t wave = std::max<int64_t>(1, (tiles + kNormBlocks - 1) / kNormBlocks);
    plan->run = (int32_t)(wave <= kNormOneWave ? wave : kNormRun);
    plan->cap = n <= kRangesSmall ? kRangesSmall : n <= kRangesMedium ? kRangesMedium : kRangesLarge;
    if (plan->cap == kRangesSmall) fill_tables(ranges, n, ranks, kNormTile, plan->run, &plan->small, &plan->rank_first);
    else if (plan->cap == kRangesMedium)
        fill_tables(ranges, n, ranks, kNormTile, plan->run, &plan->medium, &plan->rank_first);
    else {
        int64_t bytes = 0;
        for (int64_t i = 0; i < n; ++i) bytes += ranges[i].bytes;
        if (table_on_device((n + kRangesLarge - 1) / kRangesLarge, bytes)) fill_device(ranges, n, ranks, plan.get());
        else fill_tables(ranges, n, ranks, kNormTile, plan->run, &plan->large, &plan->rank_first);
    }
    if (n > 0 && plan->cap != kRangesLarge && ranks <= kFinishRanks &&
        *std::max_element(warp_tiles.begin(), warp_tiles.end()) <= kSmallTiles) {
        if (plan->cap == kRangesSmall) fill_tables(ranges, n, ranks, kWarpTile, 1, &plan->tiny_small, &plan->tiny_first);
        else fill_tables(ranges, n, ranks, kWarpTile, 1, &plan->tiny_medium, &plan->tiny_first);
    }
    return plan;
}

// Writes a chunk of a table, which is a parameter, to device memory: unlike a
// copy from host memory it can be captured, and nothing of the host has to
// outlive the call.
struct TableChunk {
    int32_t vectors;
    uint4 data[2040];
};
static_assert(sizeof(TableChunk) + 16 <= kMaxParamBytes, "table chunk exceeds the kernel parameter limit");
__global__ void __launch_bounds__(kThreads) k_upload_table(const __grid_constant__ TableChunk c, uint4* to) {
    pdl_release();
    pdl_acquire();
    for (int i = threadIdx.x; i < c.vectors; i += kThreads) to[i] = c.data[i];
}

cudaError_t upload_table(const DeviceTable& t, void* device, cudaStream_t st) {
    const int64_t all = (int64_t)t.image.size() / 16;
    uint4* to = static_cast<uint4*>(device);
    TableChunk c;
    for (int64_t i = 0; i < all; i += 2040) {
        c.vectors = (int32_t)std::min<int64_t>(2040, all - i);
        std::copy_n(t.image.data() + 16 * i, 16 * (size_t)c.vectors, reinterpret_cast<char*>(c.data));
        uint4* const at = to + i;
        const cudaError_t e = launch_table(k_upload_table, dim3(1), dim3(kThreads), st, c, at);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Where `tile`, which belongs to range i, starts in memory.
template <int64_t TILE = kNormTile, class TAB>
__device__ __forceinline__ uintptr_t tile_base(const TAB& b, int i, int tile) {
    return (reinterpret_cast<uintptr_t>(b.range[i].ptr) & ~(uintptr_t)(kNormAlign - 1)) +
           (uintptr_t)(tile - b.range[i].first) * TILE;
}

// The vector at address a, zeros where it lies outside [p, end).  A plain load,
// not a streaming one: a clip that follows finds the gradients' end in L2.
template <class E>
__device__ __forceinline__ typename E::V load_inside(uintptr_t a, uintptr_t p, uintptr_t end) {
    using V = typename E::V;
    using S = typename E::S;
    if (a >= p && a + 16 <= end) return *reinterpret_cast<const V*>(a);
    V v = make_zero<V>();
    if (a < end && a + 16 > p) {
        S* s = reinterpret_cast<S*>(&v);
#pragma unroll
        for (int l = 0; l < E::L; ++l) {
            const uintptr_t q = a + l * sizeof(S);
            if (q >= p && q < end) s[l] = *reinterpret_cast<const S*>(q);
        }
    }
    return v;
}

// The sum of squares of a thread's vectors, as four chains, which are a quarter
// as long and overlap.
template <class E, int U>
__device__ __forceinline__ float sum_squares(const typename E::V (&x)[U]) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int l = 0; l < E::L; ++l) s[l & 3] = fmaf(f32_of(x[u], l), f32_of(x[u], l), s[l & 3]);
    return (s[0] + s[1]) + (s[2] + s[3]);
}
// Zero if all of them are zeros of either sign.
template <class E, int U>
__device__ __forceinline__ uint32_t magnitude_bits(const typename E::V (&x)[U]) {
    uint32_t bits = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint4 w = *reinterpret_cast<const uint4*>(&x[u]);
        bits |= w.x | w.y | w.z | w.w;
    }
    return bits & (E::L == 8 ? 0x7FFF7FFFu : 0x7FFFFFFFu);
}

// Thread t's vectors of a tile that T threads share.
template <class E, int T>
__device__ __forceinline__ void load_tile(typename E::V (&x)[kNormVecs], int t, uintptr_t base, uintptr_t p, uintptr_t end) {
#pragma unroll
    for (int u = 0; u < kNormVecs; ++u) x[u] = load_inside<E>(base + (u * T + t) * 16, p, end);
}

// Thread t's part of a tile's sum of squares.  Where it leaves binary32's range
// and the values are not all zeros, they are loaded once more and squared
// scaled: keeping them for that would cost every tile registers.
template <class E, int T>
__device__ __forceinline__ double tile_squares(const typename E::V (&x)[kNormVecs], int t, uintptr_t base, uintptr_t p,
                                               uintptr_t end) {
    const float s = sum_squares<E>(x);
    if (in_square_range(s)) return (double)s;
    if (magnitude_bits<E>(x) == 0) return 0.0;
    WideSquares w[2];
#pragma unroll 1
    for (int u = 0; u < kNormVecs; ++u) {
        const typename E::V v = load_inside<E>(base + (u * T + t) * 16, p, end);
#pragma unroll
        for (int l = 0; l < E::L; ++l) w[l & 1].add(f32_of(v, l));
    }
    return total(w[0], w[1]);
}

// HBM bounds it: one read of every gradient, 7.58 TB/s on 8 ranks x 355M fp32
// (1.50 ms).  A thread adds a tile's squares in binary32 and the tiles in
// binary64; the block joins its threads' totals, rounded to binary32, once a
// run.  32 registers, so that eight
// blocks an SM keep 128 KB of loads in flight: bf16 took 57 with the squares'
// second pass inlined, and 112 instead of 102 us for 355M.
template <class E, class TAB>
__global__ void __launch_bounds__(kThreads, 8) k_norm_partials(const __grid_constant__ TAB b, double* partials,
                                                            const __grid_constant__ NormFinish finish) {
    __shared__ SquareScratch scratch;
    __shared__ int slot;
    init_squares(scratch);
    AcquireOnce acquire;
    pdl_release();
    if constexpr (TAB::kDevice) acquire();
    const int runs = b.tiles / b.run;
    for (int r = blockIdx.x; r < runs; r += gridDim.x) {
        int tile = r * b.run;
        int i = block_first_past(b.tile_end, b.n, tile, &slot);
        double d = 0.0;
#pragma unroll 1
        for (const int stop = tile + b.run; tile < stop; ++tile) {
            while (tile >= b.tile_end[i]) ++i;
            const uintptr_t base = tile_base(b, i, tile);
            const uintptr_t p = reinterpret_cast<uintptr_t>(b.range[i].ptr), end = p + (uintptr_t)b.range[i].bytes;
            acquire();
            typename E::V x[kNormVecs];
            load_tile<E, kThreads>(x, threadIdx.x, base, p, end);
            d += tile_squares<E, kThreads>(x, threadIdx.x, base, p, end);
        }
        const double t = block_squares((float)d, d != 0.0, scratch, [&] { return d; });
        if (threadIdx.x == 0) partials[r] = t;
        __syncthreads();                         // scratch and slot are free for the next run
    }
    finish_norms<kThreads>(finish, partials, scratch.d);
}

// The first block of a cluster takes the others' values in its shared memory:
// once it runs (each block arrives when it starts, and waits for all before it
// writes), and it reads them, or ends, after sync().  Without a cluster a block
// writes to its own.
template <bool CLUSTER>
struct ClusterStart {
    bool waited = false;
    __device__ __forceinline__ ClusterStart() {
        if constexpr (CLUSTER) asm volatile("barrier.cluster.arrive;" ::: "memory");
    }
    __device__ __forceinline__ void wait() {
        if constexpr (CLUSTER) {
            if (!waited) asm volatile("barrier.cluster.wait;" ::: "memory");
            waited = true;
        }
    }
    template <class T>
    __device__ __forceinline__ T* in_first_block(T* p) const {
        if constexpr (CLUSTER) return cooperative_groups::this_cluster().map_shared_rank(p, 0);
        return p;
    }
    __device__ __forceinline__ void sync() const {
        if constexpr (CLUSTER) cooperative_groups::this_cluster().sync();
    }
};

// The norm of little data in one launch without partials: a cluster of
// kSmallParts blocks a rank, each warp of it a 2 KB tile (or a few).  What a
// call takes here is latency: the table's lines come from a cold constant cache
// and the data from L2, one after the other, so every warp does it once and at
// the same time, and the sums meet in shared memory.  (A launch of partials and
// its last block exchange theirs through L2, twice 0.7 us away: 4.8 against 2.7
// us for 21K elements in 28 tensors; from 130 tiles on it is the faster one.)
// Under a CTA cap that has no room for the clusters one block takes the parts in
// turn.
constexpr int kSmallParts = 8;
template <class E, int CAP, bool CLUSTER>
__global__ void __launch_bounds__(kThreads) k_norm_small(const __grid_constant__ RangeTab<CAP> b,
                                                         const __grid_constant__ NormFinish f) {
    __shared__ SquareScratch scratch;
    __shared__ double part[kSmallParts];
    ClusterStart<CLUSTER> cluster;
    init_squares(scratch);
    AcquireOnce acquire;
    pdl_release();
    constexpr int kPer = CLUSTER ? kSmallParts : 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int r = blockIdx.x / kPer; r < f.ranks; r += gridDim.x / kPer) {
        const int stop = f.first[r + 1];
        for (int c = blockIdx.x % kPer; c < kSmallParts; c += kPer) {
            double d = 0.0;
            constexpr int kStep = kSmallParts * (kThreads / 32);
#pragma unroll 1
            for (int tile = f.first[r] + warp * kSmallParts + c; tile < stop; tile += 2 * kStep) {
                uintptr_t base[2], p[2], end[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {    // two tiles' table lines and data at a time; none past the rank's
                    const int t = tile + k * kStep < stop ? tile + k * kStep : tile;
                    const int i = first_past(b.tile_end, b.n, t);
                    base[k] = tile_base<kWarpTile>(b, i, t);
                    p[k] = reinterpret_cast<uintptr_t>(b.range[i].ptr);
                    end[k] = tile + k * kStep < stop ? p[k] + (uintptr_t)b.range[i].bytes : p[k];
                }
                acquire();
                typename E::V x[2][kNormVecs];
#pragma unroll
                for (int k = 0; k < 2; ++k) load_tile<E, 32>(x[k], lane, base[k], p[k], end[k]);
#pragma unroll
                for (int k = 0; k < 2; ++k) d += tile_squares<E, 32>(x[k], lane, base[k], p[k], end[k]);
            }
            acquire();
            const double t = block_squares((float)d, d != 0.0, scratch, [&] { return d; });
            cluster.wait();
            if (threadIdx.x == 0) *cluster.in_first_block(&part[c]) = t;
            __syncthreads();
        }
        cluster.sync();
        if (threadIdx.x == 0 && blockIdx.x % kPer == 0) {
            double t = part[0];
            for (int q = 1; q < kSmallParts; ++q) t += part[q];
            const float norm = norm_of(t);
            for (int q = 0; q < f.copies; ++q) f.norms[r * f.copies + q] = norm;
        }
        __syncthreads();
    }
}

struct RankFirst {
    int32_t first[DDP_MAX_WORLD + 1];
};

// Partials to norms.  Each rank's are added in `parts` parts in binary64: each
// thread's in order, then the threads' sums, then the parts'.  One block reads
// some 100 GB/s, so that the 350 thousand partials of a 355M-parameter sync
// would take it 30 us: there the parts are a cluster's blocks.  Under a CTA cap
// that has no room for them one block takes the parts in turn.
constexpr int kFinalThreads = 512;
constexpr int kFinalParts = 8;
template <bool CLUSTER>
__global__ void __launch_bounds__(kFinalThreads) k_norm_final(const double* partials, const __grid_constant__ RankFirst rf,
                                                              float* norms, int ranks, int copies, int parts) {
    __shared__ double sh[kFinalThreads / 32];
    __shared__ double part[kFinalParts];
    ClusterStart<CLUSTER> cluster;
    pdl_release();
    pdl_acquire();
    const int per = CLUSTER ? parts : 1;
    const int step = parts * kFinalThreads;
    for (int r = blockIdx.x / per; r < ranks; r += gridDim.x / per) {
        const int end = rf.first[r + 1];
        for (int c = blockIdx.x % per; c < parts; c += per) {
            double d[4] = {0.0, 0.0, 0.0, 0.0};  // four loads in flight
            int k = rf.first[r] + c * kFinalThreads + (int)threadIdx.x;
            for (; k + 3 * step < end; k += 4 * step)
#pragma unroll
                for (int u = 0; u < 4; ++u) d[u] += partials[k + u * step];
            for (; k < end; k += step) d[0] += partials[k];
            const double t = block_sum(warp_sum((d[0] + d[1]) + (d[2] + d[3])), sh);
            cluster.wait();
            if (threadIdx.x == 0) *cluster.in_first_block(&part[c]) = t;
            __syncthreads();
        }
        cluster.sync();
        if (threadIdx.x == 0 && blockIdx.x % per == 0) {
            double t = part[0];
            for (int q = 1; q < parts; ++q) t += part[q];
            for (int q = 0; q < copies; ++q) norms[r * copies + q] = norm_of(t);
        }
        __syncthreads();
    }
}

// min(1, max_norm / (norm + 1e-6)); a NaN stays one.
__device__ __forceinline__ float clip_factor(float norm, float max_norm) {
    const float c = __fdiv_rn(max_norm, norm + 1e-6f);
    return c >= 1.f ? 1.f : c;
}

__device__ __forceinline__ float scale_s(float x, float c) { return __fmul_rn(x, c); }
__device__ __forceinline__ uint16_t scale_s(uint16_t x, float c) { return f32_to_bf16_rn(__fmul_rn(bf16_to_f32(x), c)); }
__device__ __forceinline__ float4 scale_v(float4 x, float c) {
    return make_float4(__fmul_rn(x.x, c), __fmul_rn(x.y, c), __fmul_rn(x.z, c), __fmul_rn(x.w, c));
}
__device__ __forceinline__ uint32_t scale_2(uint32_t w, float c) {
    return bf16x2_rn(__fmul_rn(bf16_lo(w), c), __fmul_rn(bf16_hi(w), c));
}
__device__ __forceinline__ uint4 scale_v(uint4 x, float c) {
    return make_uint4(scale_2(x.x, c), scale_2(x.y, c), scale_2(x.z, c), scale_2(x.w, c));
}

// HBM bounds it: one read and one write of every gradient.  From the last tile
// to the first, so that the tiles a norm read last are taken from L2 (norm and
// clip of 400 MB: 181 against 186 us).
template <class E, class TAB>
__global__ void __launch_bounds__(kThreads) k_clip(const __grid_constant__ TAB b, const float* norms, float max_norm) {
    using V = typename E::V;
    using S = typename E::S;
    __shared__ int slot;
    AcquireOnce acquire;
    pdl_release();
    if constexpr (TAB::kDevice) acquire();
    for (int k = blockIdx.x; k < b.tiles; k += gridDim.x) {
        if (k != (int)blockIdx.x) __syncthreads();             // slot is free for this tile
        const int tile = b.tiles - 1 - k;
        const int i = block_first_past(b.tile_end, b.n, tile, &slot);
        const uintptr_t base = tile_base(b, i, tile);
        acquire();
        const float c = clip_factor(norms[b.range[i].rank], max_norm);
        if (c == 1.f) continue;                  // the gradients keep their bits
        const uintptr_t p = reinterpret_cast<uintptr_t>(b.range[i].ptr), end = p + (uintptr_t)b.range[i].bytes;
        V x[kNormVecs];
#pragma unroll
        for (int u = 0; u < kNormVecs; ++u) {
            const uintptr_t a = base + (u * kThreads + threadIdx.x) * 16;
            if (a >= p && a + 16 <= end) x[u] = ld_stream<V>(reinterpret_cast<const void*>(a));
        }
#pragma unroll
        for (int u = 0; u < kNormVecs; ++u) {
            const uintptr_t a = base + (u * kThreads + threadIdx.x) * 16;
            if (a >= p && a + 16 <= end) {
                st_stream<V>(reinterpret_cast<void*>(a), scale_v(x[u], c));
            } else if (a < end && a + 16 > p) {
                for (int l = 0; l < E::L; ++l) {
                    S* q = reinterpret_cast<S*>(a + l * sizeof(S));
                    if (reinterpret_cast<uintptr_t>(q) >= p && reinterpret_cast<uintptr_t>(q) < end) *q = scale_s(*q, c);
                }
            }
        }
    }
}

static NormFinish finish_of(NormSpace ws, const int32_t* rank_first, int ranks, int copies, float* norms) {
    NormFinish f{};
    f.counter = ws.counter;
    f.norms = norms;
    f.ranks = ranks;
    f.copies = copies;
    std::copy(rank_first, rank_first + ranks + 1, f.first);
    return f;
}

NormFinish norm_finish(NormSpace ws, const int32_t* rank_first, int ranks, int copies, float* norms, bool one_launch) {
    if (!one_launch || ranks > kFinishRanks || rank_first[ranks] > kFinishPartials) return NormFinish{};
    return finish_of(ws, rank_first, ranks, copies, norms);
}

static bool room_for(int64_t blocks) { return cap_ctas(blocks) == blocks; }

template <class E, int CAP>
static cudaError_t norm_small(const RangeTab<CAP>& b, const NormFinish& f, cudaStream_t st) {
    if (room_for(f.ranks * kSmallParts))
        return launch_table<kSmallParts>(k_norm_small<E, CAP, true>, dim3(f.ranks * kSmallParts), dim3(kThreads), st, b, f);
    return launch_table(k_norm_small<E, CAP, false>, dim3(cap_ctas(f.ranks)), dim3(kThreads), st, b, f);
}

template <class E, class TAB>
static cudaError_t norm_table(const TAB& b, double* partials, const NormFinish& finish, cudaStream_t st) {
    return launch_table(k_norm_partials<E, TAB>, dim3(cap_ctas(b.tiles / b.run)), dim3(kThreads), st, b, partials, finish);
}

template <class E, class TAB>
static cudaError_t norm_tables(const std::vector<TAB>& tables, double* partials, const NormFinish& finish,
                               cudaStream_t st) {
    for (const TAB& b : tables) {
        const cudaError_t e = norm_table<E>(b, partials, finish, st);
        if (e != cudaSuccess) return e;
        partials += b.tiles / b.run;
    }
    return cudaSuccess;
}

template <class E>
static cudaError_t norm_kernels(const RangePlan& plan, NormSpace ws, int copies, float* norms, cudaStream_t st) {
    const int ranks = (int)plan.rank_first.size() - 1;
    const int32_t* first = plan.rank_first.data();
    if (!plan.tiny_first.empty()) {
        const NormFinish f = finish_of(ws, plan.tiny_first.data(), ranks, copies, norms);
        if (plan.cap == kRangesSmall) return norm_small<E>(plan.tiny_small[0], f, st);
        return norm_small<E>(plan.tiny_medium[0], f, st);
    }
    const bool device = !plan.device.image.empty();
    const size_t launches = plan.small.size() + plan.medium.size() + plan.large.size() + (device ? 1 : 0);
    const NormFinish f = norm_finish(ws, first, ranks, copies, norms, launches == 1);
    cudaError_t e;
    if (device) e = norm_table<E>(device_ranges(plan, ws.table), ws.partials, f, st);
    else if (plan.cap == kRangesSmall) e = norm_tables<E>(plan.small, ws.partials, f, st);
    else if (plan.cap == kRangesMedium) e = norm_tables<E>(plan.medium, ws.partials, f, st);
    else e = norm_tables<E>(plan.large, ws.partials, f, st);
    if (e != cudaSuccess || f.counter) return e;
    return launch_norm_final(ws.partials, first, ranks, copies, norms, st);
}

cudaError_t launch_norm(const RangePlan& plan, int dtype, NormSpace ws, int copies, float* norms, cudaStream_t st) {
    return dtype == DDP_BF16 ? norm_kernels<EBF16>(plan, ws, copies, norms, st)
                             : norm_kernels<EF32>(plan, ws, copies, norms, st);
}

cudaError_t launch_norm_final(const double* partials, const int32_t* rank_first, int ranks, int copies, float* norms,
                              cudaStream_t st) {
    RankFirst rf;
    std::copy(rank_first, rank_first + ranks + 1, rf.first);
    int32_t most = 0;
    for (int r = 0; r < ranks; ++r) most = std::max(most, rank_first[r + 1] - rank_first[r]);
    const int parts = most <= 8 * kFinalThreads ? 1 : kFinalParts;
    if (parts > 1 && room_for((int64_t)ranks * parts))
        return launch_table<kFinalParts>(k_norm_final<true>, dim3(ranks * parts), dim3(kFinalThreads), st, partials, rf,
                                         norms, ranks, copies, parts);
    return launch_table(k_norm_final<false>, dim3(cap_ctas(ranks)), dim3(kFinalThreads), st, partials, rf, norms, ranks,
                        copies, parts);
}

template <class E, class TAB>
static cudaError_t clip_table(const TAB& b, const float* norms, float max_norm, cudaStream_t st) {
    return launch_table(k_clip<E, TAB>, dim3(cap_ctas(b.tiles)), dim3(kThreads), st, b, norms, max_norm);
}

template <class E, class TAB>
static cudaError_t clip_tables(const std::vector<TAB>& tables, const float* norms, float max_norm, cudaStream_t st) {
    for (const TAB& b : tables) {
        const cudaError_t e = clip_table<E>(b, norms, max_norm, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <class E>
static cudaError_t clip(const RangePlan& plan, NormSpace ws, const float* norms, float max_norm, cudaStream_t st) {
    if (!plan.device.image.empty()) return clip_table<E>(device_ranges(plan, ws.table), norms, max_norm, st);
    if (plan.cap == kRangesSmall) return clip_tables<E>(plan.small, norms, max_norm, st);
    if (plan.cap == kRangesMedium) return clip_tables<E>(plan.medium, norms, max_norm, st);
    return clip_tables<E>(plan.large, norms, max_norm, st);
}

cudaError_t launch_clip(const RangePlan& plan, int dtype, NormSpace ws, const float* norms, float max_norm,
                        cudaStream_t st) {
    return dtype == DDP_BF16 ? clip<EBF16>(plan, ws, norms, max_norm, st) : clip<EF32>(plan, ws, norms, max_norm, st);
}

}  // namespace ddpk
