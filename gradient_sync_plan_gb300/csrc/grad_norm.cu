// grad_norm.cu -- the global gradient norm over many tensors, and clipping.
//
//   norms[r] = sqrt(sum over rank r's tensors and elements of g^2)
//   g <- c g,  c = min(1, max_norm / (norms[r] + 1e-6)),  rounded once to g's type
//
// Both walk a table of byte ranges (tensors that lie back to back are one),
// cut into tiles at 128-byte boundaries of memory: every 16-byte access is
// aligned wherever a tensor starts, and only a range's first and last vector
// are taken element by element.  The table travels in the kernel's parameters.
// A tile's partial sum depends on the tile alone and the partials are added in
// a fixed order, so a norm does not depend on the grid that computed it.
#include <cooperative_groups.h>

#include <algorithm>
#include <climits>

#include "norm_device.cuh"
#include "optim_internal.h"

namespace ddpk {

template <int CAP>
struct RangeTab {
    int32_t n;
    int32_t tiles;
    char* ptr[CAP];
    int64_t bytes[CAP];
    int32_t tile_end[CAP];     // inclusive prefix of tiles
    int32_t rank[CAP];
};
constexpr int kRangesSmall = 32;
constexpr int kRangesLarge = 1280;
static_assert(sizeof(RangeTab<kRangesLarge>) + 64 <= kMaxParamBytes, "range table exceeds the kernel parameter limit");

int64_t range_tiles(const void* ptr, int64_t bytes) {
    const int64_t lead = (int64_t)(reinterpret_cast<uintptr_t>(ptr) % kNormAlign);
    return (lead + bytes + kNormTile - 1) / kNormTile;
}

// The range that holds `tile`, and where the tile starts in memory.
template <int CAP>
__device__ __forceinline__ int range_of(const RangeTab<CAP>& b, int tile, uintptr_t* base) {
    const int lo = first_past(b.tile_end, b.n, tile);
    const int first = lo ? b.tile_end[lo - 1] : 0;
    *base = (reinterpret_cast<uintptr_t>(b.ptr[lo]) & ~(uintptr_t)(kNormAlign - 1)) + (uintptr_t)(tile - first) * kNormTile;
    return lo;
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

template <class E, int CAP>
__global__ void __launch_bounds__(kThreads) k_norm_partials(const __grid_constant__ RangeTab<CAP> b, double* partials) {
    __shared__ double sh[kThreads / 32];
    pdl_release();
    pdl_acquire();
    for (int tile = blockIdx.x; tile < b.tiles; tile += gridDim.x) {
        uintptr_t base;
        const int i = range_of(b, tile, &base);
        const uintptr_t p = reinterpret_cast<uintptr_t>(b.ptr[i]), end = p + (uintptr_t)b.bytes[i];
        typename E::V x[kNormVecs];
#pragma unroll
        for (int u = 0; u < kNormVecs; ++u) x[u] = load_inside<E>(base + (u * kThreads + threadIdx.x) * 16, p, end);
        const double t = block_sum(warp_sum_squares<E>(x), sh);
        if (threadIdx.x == 0) partials[tile] = t;
        __syncthreads();                         // sh is free for the next tile
    }
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
        for (int q = 0; q < copies; ++q) norms[r * copies + q] = (float)sqrt(t);
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
    pdl_release();
    pdl_acquire();
    for (int tile = blockIdx.x; tile < b.tiles; tile += gridDim.x) {
        uintptr_t base;
        const int i = range_of(b, tile, &base);
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

// Fill tables with consecutive ranges and hand each to launch(table, tiles before it).
template <int CAP, class Launch>
static cudaError_t for_tables(const GradRange* ranges, int64_t n, Launch launch) {
    RangeTab<CAP> b;
    int64_t i = 0, before = 0;
    while (i < n) {
        b.n = 0;
        b.tiles = 0;
        for (; i < n && b.n < CAP; ++i, ++b.n) {
            b.tiles += (int32_t)range_tiles(ranges[i].ptr, ranges[i].bytes);
            b.ptr[b.n] = ranges[i].ptr;
            b.bytes[b.n] = ranges[i].bytes;
            b.tile_end[b.n] = b.tiles;
            b.rank[b.n] = ranges[i].rank;
        }
        const cudaError_t e = launch(b, before);
        if (e != cudaSuccess) return e;
        before += b.tiles;
    }
    return cudaSuccess;
}

template <class E, int CAP>
static cudaError_t norm_partials(const GradRange* ranges, int64_t n, double* partials, cudaStream_t st) {
    return for_tables<CAP>(ranges, n, [&](const RangeTab<CAP>& b, int64_t before) {
        return launch_dependent(k_norm_partials<E, CAP>, dim3(cap_ctas(b.tiles)), dim3(kThreads), 0, st, b,
                                partials + before);
    });
}

template <class E, int CAP>
static cudaError_t clip(const GradRange* ranges, int64_t n, const float* norms, float max_norm, cudaStream_t st) {
    return for_tables<CAP>(ranges, n, [&](const RangeTab<CAP>& b, int64_t) {
        return launch_dependent(k_clip<E, CAP>, dim3(cap_ctas(b.tiles)), dim3(kThreads), 0, st, b, norms, max_norm);
    });
}

cudaError_t launch_norm_partials(const GradRange* ranges, int64_t n, int dtype, double* partials, cudaStream_t st) {
    if (n <= kRangesSmall)
        return dtype == DDP_BF16 ? norm_partials<EBF16, kRangesSmall>(ranges, n, partials, st)
                                 : norm_partials<EF32, kRangesSmall>(ranges, n, partials, st);
    return dtype == DDP_BF16 ? norm_partials<EBF16, kRangesLarge>(ranges, n, partials, st)
                             : norm_partials<EF32, kRangesLarge>(ranges, n, partials, st);
}

cudaError_t launch_norm_final(const double* partials, const int32_t* rank_first, int ranks, int copies, float* norms,
                              cudaStream_t st) {
    RankFirst rf;
    std::copy(rank_first, rank_first + ranks + 1, rf.first);
    int32_t most = 0;
    for (int r = 0; r < ranks; ++r) most = std::max(most, rank_first[r + 1] - rank_first[r]);
    if (most <= 8 * kFinalThreads)
        return launch_dependent(k_norm_final<1>, dim3(ranks), dim3(kFinalThreads), 0, st, partials, rf, norms, copies);
    return launch_cluster<kFinalBlocks>(k_norm_final<kFinalBlocks>, dim3(ranks * kFinalBlocks), dim3(kFinalThreads), st,
                                        partials, rf, norms, copies);
}

cudaError_t launch_clip(const GradRange* ranges, int64_t n, int dtype, const float* norms, float max_norm,
                        cudaStream_t st) {
    if (n <= kRangesSmall)
        return dtype == DDP_BF16 ? clip<EBF16, kRangesSmall>(ranges, n, norms, max_norm, st)
                                 : clip<EF32, kRangesSmall>(ranges, n, norms, max_norm, st);
    return dtype == DDP_BF16 ? clip<EBF16, kRangesLarge>(ranges, n, norms, max_norm, st)
                             : clip<EF32, kRangesLarge>(ranges, n, norms, max_norm, st);
}

}  // namespace ddpk
