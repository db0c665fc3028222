// grad_norm.cu -- the global gradient norm over many tensors, and clipping.
//
//   norms[r] = sqrt(sum over rank r's tensors and elements of g^2)
//   g <- c g,  c = min(1, max_norm / (norms[r] + 1e-6)),  rounded once to g's type
//
// Both walk a table of byte ranges (tensors that lie back to back are one),
// cut into tiles at 128-byte boundaries of memory: every 16-byte access is
// aligned wherever a tensor starts, and only a range's first and last vector
// are taken element by element.  The tables are filled once and travel in the
// kernels' parameters.  A norm block takes a run of up to four tiles and leaves
// one partial sum; runs depend on the tensors alone and partials are added in a
// fixed order, so a norm does not depend on the grid that computed it.
#include <cooperative_groups.h>

#include <algorithm>
#include <climits>

#include "norm_device.cuh"
#include "optim_internal.h"

namespace ddpk {

template <int CAP>
struct RangeTab {
    int32_t n;
    int32_t tiles;             // a multiple of `run`
    int32_t run;               // tiles a norm block takes: never of two ranks
    char* ptr[CAP];
    int64_t bytes[CAP];
    int32_t tile_end[CAP];     // inclusive prefix of tiles; a rank's last range has the padding to a whole run
    int32_t rank[CAP];
};
// Capacities: a launch's parameters are copied for every eager launch.
constexpr int kRangesSmall = 32;
constexpr int kRangesMedium = 320;
constexpr int kRangesLarge = 1280;
static_assert(sizeof(RangeTab<kRangesLarge>) + sizeof(NormFinish) + 64 <= kMaxParamBytes,
              "range table exceeds the kernel parameter limit");

struct RangePlan {
    int cap = 0;
    std::vector<RangeTab<kRangesSmall>> small;
    std::vector<RangeTab<kRangesMedium>> medium;
    std::vector<RangeTab<kRangesLarge>> large;
    int32_t run = 1;
    std::vector<int32_t> rank_first;             // first partial of each rank, and their end
};

static int64_t range_tiles(const GradRange& g) {
    const int64_t lead = (int64_t)(reinterpret_cast<uintptr_t>(g.ptr) % kNormAlign);
    return (lead + g.bytes + kNormTile - 1) / kNormTile;
}

template <int CAP>
static void fill_tables(const GradRange* ranges, int64_t n, int ranks, RangePlan* plan, std::vector<RangeTab<CAP>>* out) {
    plan->cap = CAP;
    plan->rank_first.assign(ranks + 1, 0);
    int64_t partials = 0;
    int rank = 0;                                // ranks below it have their rank_first
    for (int64_t i = 0; i < n;) {
        out->emplace_back();
        RangeTab<CAP>& b = out->back();
        b.n = 0;
        b.run = plan->run;
        int64_t tiles = 0;
        for (; i < n && b.n < CAP; ++i, ++b.n) {
            while (rank < ranges[i].rank) plan->rank_first[++rank] = (int32_t)(partials + tiles / plan->run);
            tiles += range_tiles(ranges[i]);
            if (b.n + 1 == CAP || i + 1 == n || ranges[i + 1].rank != ranges[i].rank)
                tiles = (tiles + plan->run - 1) / plan->run * plan->run;
            b.ptr[b.n] = ranges[i].ptr;
            b.bytes[b.n] = ranges[i].bytes;
            b.tile_end[b.n] = (int32_t)tiles;
            b.rank[b.n] = ranges[i].rank;
        }
        b.tiles = (int32_t)tiles;
        partials += tiles / plan->run;
    }
    while (rank < ranks) plan->rank_first[++rank] = (int32_t)partials;
}

std::shared_ptr<const RangePlan> make_range_plan(const GradRange* ranges, int64_t n, int ranks) {
    auto plan = std::make_shared<RangePlan>();
    int64_t tiles = 0;
    for (int64_t i = 0; i < n; ++i) tiles += range_tiles(ranges[i]);
    // one wave of eight blocks an SM while a run of four is enough for that
    plan->run = (int32_t)std::min<int64_t>(kNormRun, std::max<int64_t>(1, (tiles + kNormBlocks - 1) / kNormBlocks));
    if (n <= kRangesSmall) fill_tables(ranges, n, ranks, plan.get(), &plan->small);
    else if (n <= kRangesMedium) fill_tables(ranges, n, ranks, plan.get(), &plan->medium);
    else fill_tables(ranges, n, ranks, plan.get(), &plan->large);
    return plan;
}

int64_t range_plan_partials(const RangePlan& plan) { return plan.rank_first.back(); }

// Where `tile`, which belongs to range i, starts in memory.
template <int CAP>
__device__ __forceinline__ uintptr_t tile_base(const RangeTab<CAP>& b, int i, int tile) {
    const int first = i ? b.tile_end[i - 1] : 0;
    return (reinterpret_cast<uintptr_t>(b.ptr[i]) & ~(uintptr_t)(kNormAlign - 1)) + (uintptr_t)(tile - first) * kNormTile;
}

// The vector at address a, zeros where it lies outside [p, end).
template <class E>
__device__ __forceinline__ typename E::V load_inside(uintptr_t a, uintptr_t p, uintptr_t end) {
    using V = typename E::V;
    using S = typename E::S;
    if (a >= p && a + 16 <= end) return ld_stream<V>(reinterpret_cast<const void*>(a));
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

constexpr int kNormVecs = (int)(kNormTile / 16 / kThreads);      // vectors a thread takes of a tile

// The sum of squares of a thread's vectors: in binary32 as four chains, which
// are a quarter as long and overlap; in binary64 where that leaves its range.
template <class E, int U>
__device__ __forceinline__ float sum_squares(const typename E::V (&x)[U]) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int l = 0; l < E::L; ++l) s[l & 3] = fmaf(f32_of(x[u], l), f32_of(x[u], l), s[l & 3]);
    return (s[0] + s[1]) + (s[2] + s[3]);
}
template <class E, int U>
__device__ __forceinline__ double sum_squares64(const typename E::V (&x)[U]) {
    double d = 0.0;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int l = 0; l < E::L; ++l) d = fma((double)f32_of(x[u], l), (double)f32_of(x[u], l), d);
    return d;
}
// Whether any of them is not a zero of either sign.
template <class E, int U>
__device__ __forceinline__ bool any_nonzero(const typename E::V (&x)[U]) {
    uint32_t bits = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint4 w = *reinterpret_cast<const uint4*>(&x[u]);
        bits |= w.x | w.y | w.z | w.w;
    }
    return (bits & (E::L == 8 ? 0x7FFF7FFFu : 0x7FFFFFFFu)) != 0;
}

// HBM bounds it: one read of every gradient.  A thread adds a tile's squares in
// binary32 and the tiles in binary64; the block joins its threads once a run.
template <class E, int CAP>
__global__ void __launch_bounds__(kThreads) k_norm_partials(const __grid_constant__ RangeTab<CAP> b, double* partials,
                                                            const __grid_constant__ NormFinish finish) {
    __shared__ SquareScratch scratch;
    __shared__ int slot;
    init_squares(scratch);
    pdl_release();
    pdl_acquire();
    const int runs = b.tiles / b.run;
    for (int r = blockIdx.x; r < runs; r += gridDim.x) {
        int tile = r * b.run;
        int i = block_first_past(b.tile_end, b.n, tile, &slot);
        double d = 0.0;
#pragma unroll 1
        for (const int stop = tile + b.run; tile < stop; ++tile) {
            while (tile >= b.tile_end[i]) ++i;
            const uintptr_t base = tile_base(b, i, tile);
            const uintptr_t p = reinterpret_cast<uintptr_t>(b.ptr[i]), end = p + (uintptr_t)b.bytes[i];
            typename E::V x[kNormVecs];
#pragma unroll
            for (int u = 0; u < kNormVecs; ++u) x[u] = load_inside<E>(base + (u * kThreads + threadIdx.x) * 16, p, end);
            const float s = sum_squares<E>(x);
            if (in_square_range(s)) d += (double)s;
            else if (any_nonzero<E>(x)) d += sum_squares64<E>(x);
        }
        const double t = block_squares((float)d, d != 0.0, scratch, [&] { return d; });
        if (threadIdx.x == 0) partials[r] = t;
        __syncthreads();                         // scratch and slot are free for the next run
    }
    finish_norms<kThreads>(finish, partials, scratch.d);
}

struct RankFirst {
    int32_t first[DDP_MAX_WORLD + 1];
};

// A cluster of C blocks a rank: its partials added in binary64, each thread's
// in order, then the threads' sums, then the blocks'.  One block reads some
// 100 GB/s, so that the 350 thousand partials of a 355M-parameter sync would
// take it 30 us; eight share them.
constexpr int kFinalThreads = 512;
constexpr int kFinalBlocks = 8;
template <int C>
__global__ void __launch_bounds__(kFinalThreads) k_norm_final(const double* partials, const __grid_constant__ RankFirst rf,
                                                              float* norms, int copies) {
    __shared__ double sh[kFinalThreads / 32];
    __shared__ double block[C];
    pdl_release();
    pdl_acquire();
    const int r = blockIdx.x / C, c = blockIdx.x % C;
    const int end = rf.first[r + 1];
    constexpr int kStep = C * kFinalThreads;
    double d[4] = {0.0, 0.0, 0.0, 0.0};          // four loads in flight
    int k = rf.first[r] + c * kFinalThreads + (int)threadIdx.x;
    for (; k + 3 * kStep < end; k += 4 * kStep)
#pragma unroll
        for (int u = 0; u < 4; ++u) d[u] += partials[k + u * kStep];
    for (; k < end; k += kStep) d[0] += partials[k];
    double t = block_sum(warp_sum((d[0] + d[1]) + (d[2] + d[3])), sh);
    if constexpr (C > 1) {
        auto cluster = cooperative_groups::this_cluster();
        if (threadIdx.x == 0) cluster.map_shared_rank(block, 0)[c] = t;
        cluster.sync();
        if (threadIdx.x == 0 && c == 0) {
            t = block[0];
            for (int q = 1; q < C; ++q) t += block[q];
        }
    }
    if (threadIdx.x == 0 && c == 0)
        for (int q = 0; q < copies; ++q) norms[r * copies + q] = norm_of(t);
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

template <class E, int CAP>
__global__ void __launch_bounds__(kThreads) k_clip(const __grid_constant__ RangeTab<CAP> b, const float* norms, float max_norm) {
    using V = typename E::V;
    using S = typename E::S;
    __shared__ int slot;
    pdl_release();
    pdl_acquire();
    for (int tile = blockIdx.x; tile < b.tiles; tile += gridDim.x) {
        if (tile != (int)blockIdx.x) __syncthreads();          // slot is free for this tile
        const int i = block_first_past(b.tile_end, b.n, tile, &slot);
        const uintptr_t base = tile_base(b, i, tile);
        const float c = clip_factor(norms[b.rank[i]], max_norm);
        if (c == 1.f) continue;                  // the gradients keep their bits
        const uintptr_t p = reinterpret_cast<uintptr_t>(b.ptr[i]), end = p + (uintptr_t)b.bytes[i];
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

NormFinish norm_finish(NormSpace ws, const int32_t* rank_first, int ranks, int copies, float* norms, bool one_launch) {
    NormFinish f{};
    if (!one_launch || ranks > kFinishRanks || rank_first[ranks] > kFinishPartials) return f;
    f.counter = ws.counter;
    f.norms = norms;
    f.ranks = ranks;
    f.copies = copies;
    std::copy(rank_first, rank_first + ranks + 1, f.first);
    return f;
}

template <class E, int CAP>
static cudaError_t norm_tables(const std::vector<RangeTab<CAP>>& tables, double* partials, const NormFinish& finish,
                               cudaStream_t st) {
    for (const RangeTab<CAP>& b : tables) {
        const int runs = b.tiles / b.run;
        const cudaError_t e = launch_table(k_norm_partials<E, CAP>, dim3(cap_ctas(runs)), dim3(kThreads), st, b, partials,
                                           finish);
        if (e != cudaSuccess) return e;
        partials += runs;
    }
    return cudaSuccess;
}

template <class E>
static cudaError_t norm_partials(const RangePlan& plan, double* partials, const NormFinish& f, cudaStream_t st) {
    if (plan.cap == kRangesSmall) return norm_tables<E>(plan.small, partials, f, st);
    if (plan.cap == kRangesMedium) return norm_tables<E>(plan.medium, partials, f, st);
    return norm_tables<E>(plan.large, partials, f, st);
}

cudaError_t launch_norm(const RangePlan& plan, int dtype, NormSpace ws, int copies, float* norms, cudaStream_t st) {
    const int ranks = (int)plan.rank_first.size() - 1;
    const size_t launches = plan.small.size() + plan.medium.size() + plan.large.size();
    const NormFinish f = norm_finish(ws, plan.rank_first.data(), ranks, copies, norms, launches == 1);
    const cudaError_t e = dtype == DDP_BF16 ? norm_partials<EBF16>(plan, ws.partials, f, st)
                                            : norm_partials<EF32>(plan, ws.partials, f, st);
    if (e != cudaSuccess || f.counter) return e;
    return launch_norm_final(ws.partials, plan.rank_first.data(), ranks, copies, norms, st);
}

cudaError_t launch_norm_final(const double* partials, const int32_t* rank_first, int ranks, int copies, float* norms,
                              cudaStream_t st) {
    RankFirst rf;
    std::copy(rank_first, rank_first + ranks + 1, rf.first);
    int32_t most = 0;
    for (int r = 0; r < ranks; ++r) most = std::max(most, rank_first[r + 1] - rank_first[r]);
    if (most <= 8 * kFinalThreads)
        return launch_table(k_norm_final<1>, dim3(ranks), dim3(kFinalThreads), st, partials, rf, norms, copies);
    return launch_table<kFinalBlocks>(k_norm_final<kFinalBlocks>, dim3(ranks * kFinalBlocks), dim3(kFinalThreads), st,
                                      partials, rf, norms, copies);
}

template <class E, int CAP>
static cudaError_t clip_tables(const std::vector<RangeTab<CAP>>& tables, const float* norms, float max_norm,
                               cudaStream_t st) {
    for (const RangeTab<CAP>& b : tables) {
        const cudaError_t e = launch_table(k_clip<E, CAP>, dim3(cap_ctas(b.tiles)), dim3(kThreads), st, b, norms, max_norm);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <class E>
static cudaError_t clip(const RangePlan& plan, const float* norms, float max_norm, cudaStream_t st) {
    if (plan.cap == kRangesSmall) return clip_tables<E>(plan.small, norms, max_norm, st);
    if (plan.cap == kRangesMedium) return clip_tables<E>(plan.medium, norms, max_norm, st);
    return clip_tables<E>(plan.large, norms, max_norm, st);
}

cudaError_t launch_clip(const RangePlan& plan, int dtype, const float* norms, float max_norm, cudaStream_t st) {
    return dtype == DDP_BF16 ? clip<EBF16>(plan, norms, max_norm, st) : clip<EF32>(plan, norms, max_norm, st);
}

}  // namespace ddpk
