// norm_device.cuh -- sums of squares, shared by the kernels that take a norm.
//
// A thread adds the squares of its part of a tile in binary32 and, where its
// block takes several tiles for one partial sum, the tiles in binary64.  Its
// total is rounded to binary32 and the block joins its threads in binary32;
// partial sums are added in binary64.  That join is a tree of ten additions,
// less than a long chain's own error, and half the words of one in binary64.
// All terms are positive, so a partial sum's relative error stays within chain
// length + 14 units of 2^-24 (3 additions of the chains, the rounding, the
// join), and far below that on average.  The longest chain has 32 terms: a bf16
// sync with four vectors a thread that go element by element (the ranks'
// pointers lie differently against 16 bytes); elsewhere it has up to 16.  A square
// leaves binary32's range long before its value does (2^-75 squares to nothing,
// 2^64 to infinity), so a tile with a warp whose sum falls outside
// [2^-90, 2^112] squares again with scaled values, from registers or memory that
// still hold them.  Inside that range what underflow took is below 2^-136 a
// warp, nothing next to 2^-90, and 32 warps' sums stay finite.
#pragma once

#include <type_traits>

#include "ddp_device.cuh"
#include "optim_internal.h"

namespace ddpk {

// launch_dependent for a kernel whose first parameter is a table the caller
// keeps: its address goes to the launch, which copies it once.  C > 1: blocks
// form clusters of C.
template <int C = 1, class... KArgs, class... Args>
inline cudaError_t launch_table(void (*kernel)(KArgs...), dim3 grid, dim3 block, cudaStream_t st, const Args&... args) {
    static_assert(sizeof...(KArgs) == sizeof...(Args), "one argument a parameter");
    static_assert((std::is_same<KArgs, Args>::value && ...), "arguments of the parameters' own types");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 2 : 1;
    void* p[] = {const_cast<void*>(static_cast<const void*>(&args))...};
    const cudaError_t e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kernel), p);
    const cudaError_t last = cudaGetLastError();
    return e != cudaSuccess ? e : last;
}

__device__ __forceinline__ float f32_of(float4 v, int l) { return l == 0 ? v.x : l == 1 ? v.y : l == 2 ? v.z : v.w; }
__device__ __forceinline__ float f32_of(uint4 v, int l) {
    const uint32_t w = (l >> 1) == 0 ? v.x : (l >> 1) == 1 ? v.y : (l >> 1) == 2 ? v.z : v.w;
    return (l & 1) ? bf16_hi(w) : bf16_lo(w);
}

__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    return s;
}
__device__ __forceinline__ double warp_sum(double s) {
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    return s;
}

// Whether a warp's sum of squares can be trusted in binary32 (so can a zero, if
// every value is one).
__device__ __forceinline__ bool in_square_range(float w) { return w >= 0x1p-90f && w <= 0x1p112f; }

// pdl_acquire at its first call: after a block has found its place in the table,
// which is a parameter and waits for nobody, and before it touches memory.  The
// search (1 to 2 us from a cold constant cache) then overlaps the tail of the
// kernel before.
struct AcquireOnce {
    bool done = false;
    __device__ __forceinline__ void operator()() {
        if (!done) pdl_acquire();
        done = true;
    }
};

// A sum of squares of any binary32 values, in binary32 but for its end: the
// large and the small ones are scaled by a power of two before they are squared
// (2^-100 and 2^100: every finite value's square is then in range) and added
// apart.  An infinity or a NaN comes out as one.
struct WideSquares {
    float low = 0.f, mid = 0.f, high = 0.f;
    __device__ __forceinline__ void add(float f) {
        const float a = fabsf(f);
        if (a > 0x1p40f) high = fmaf(f * 0x1p-100f, f * 0x1p-100f, high);
        else if (a < 0x1p-40f) low = fmaf(f * 0x1p100f, f * 0x1p100f, low);
        else mid = fmaf(f, f, mid);
    }
};
// Two of them (half the chain each) together.
__device__ __forceinline__ double total(const WideSquares& a, const WideSquares& b) {
    return (double)(a.low + b.low) * 0x1p-200 + ((double)(a.mid + b.mid) + (double)(a.high + b.high) * 0x1p200);
}

// One value a warp -> their sum in every lane of warp 0 (undefined elsewhere).
// `sh` has a slot a warp; the caller puts a barrier between two uses.
template <class T>
__device__ __forceinline__ T block_sum(T warp_total, T* sh) {
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = warp_total;
    __syncthreads();
    T t = 0;
    if (threadIdx.x < 32) t = warp_sum((int)threadIdx.x < warps ? sh[threadIdx.x] : T(0));
    return t;
}

// Scratch of a block's sum of squares.
struct SquareScratch {
    float w[32];
    double d[32];
    int odd;                                     // some warp's sum is out of the safe range
};
__device__ __forceinline__ void init_squares(SquareScratch& sc) {
    if (threadIdx.x == 0) sc.odd = 0;
    __syncthreads();
}

// The block's sum of squares in warp 0's lanes, from each thread's own sum s in
// binary32.  Where a warp's is out of range and not all of its values are
// zeros (nonzero), every thread squares again: again() -> double.  Ends without
// a barrier; the caller puts one before the next use.
template <class Again>
__device__ __forceinline__ double block_squares(float s, bool nonzero, SquareScratch& sc, Again again) {
    const float w = warp_sum(s);
    const bool odd = !in_square_range(w) && __any_sync(0xffffffffu, nonzero);
    if ((threadIdx.x & 31) == 0) {
        sc.w[threadIdx.x >> 5] = w;
        if (odd) sc.odd = 1;
    }
    __syncthreads();
    if (!sc.odd) return threadIdx.x < 32 ? (double)warp_sum((int)threadIdx.x < (int)blockDim.x >> 5 ? sc.w[threadIdx.x] : 0.f) : 0.0;
    const double t = block_sum(warp_sum(again()), sc.d);
    if (threadIdx.x == 0) sc.odd = 0;
    return t;
}

__device__ __forceinline__ float norm_of(double squares) {
    // half a rounding more than from the binary64 root, which takes ten times as long
    if (squares >= 0x1p-120 && squares <= 0x1p120) return __fsqrt_rn((float)squares);
    return (float)sqrt(squares);
}

// The first of n ascending ends that lies past x (x is below the last end).
// Each lane looks at one entry of a stride, then at one of the stretch that is
// left: two rounds of loads for up to 1024 entries, where halving takes ten,
// one behind the other.  The whole warp must call it.
__device__ __forceinline__ int first_past(const int32_t* ends, int n, int x) {
    const int lane = threadIdx.x & 31;
    int from = 0;
    int stride = 1;
    while (stride * 32 < n) stride *= 32;
    for (;; stride /= 32) {
        const int at = min(from + (lane + 1) * stride, n) - 1;
        const unsigned past = __ballot_sync(0xffffffffu, ends[at] > x);
        from += (__ffs(past) - 1) * stride;
        if (stride == 1) return from;
    }
}

// first_past for a whole block: warp 0 looks, the others read what it found from
// `slot` (a divergent load of the table keeps the constant cache busy for 32
// accesses: one warp's is enough).  A barrier has to lie between two uses.
__device__ __forceinline__ int block_first_past(const int32_t* ends, int n, int x, int* slot) {
    if (n == 1) return 0;
    if (threadIdx.x < 32) {
        const int i = first_past(ends, n, x);
        if (threadIdx.x == 0) *slot = i;
    }
    __syncthreads();
    return *slot;
}

// The end of a launch that has all the partials: the block that arrives last
// adds each rank's in a fixed order and writes the norms.  atomicInc wraps the
// counter back to zero for the next launch.  Every thread of the block calls
// it, after its block's partials are written (by thread 0).
template <int THREADS>
__device__ __forceinline__ void finish_norms(const NormFinish& f, const double* partials, double* sh) {
    __shared__ bool last;
    if (!f.counter) return;
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicInc(f.counter, gridDim.x - 1) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    int groups = 1;                              // ranks side by side, each by a whole number of warps
    while (groups < f.ranks && groups < THREADS / 32) groups *= 2;
    const int per = THREADS / groups, g = threadIdx.x / per, t = threadIdx.x % per;
    for (int r0 = 0; r0 < f.ranks; r0 += groups) {
        const int r = r0 + g;
        const int end = r < f.ranks ? f.first[r + 1] : 0;
        double d[4] = {0.0, 0.0, 0.0, 0.0};
        int k = r < f.ranks ? f.first[r] + t : 0;
        for (; k + 3 * per < end; k += 4 * per)
#pragma unroll
            for (int u = 0; u < 4; ++u) d[u] += __ldcg(partials + k + u * per);
        for (; k < end; k += per) d[0] += __ldcg(partials + k);
        const double w = warp_sum((d[0] + d[1]) + (d[2] + d[3]));
        if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = w;
        __syncthreads();
        if (t == 0 && r < f.ranks) {
            double s = sh[threadIdx.x >> 5];
            for (int q = 1; q < per / 32; ++q) s += sh[(threadIdx.x >> 5) + q];
            const float norm = norm_of(s);
            for (int q = 0; q < f.copies; ++q) f.norms[r * f.copies + q] = norm;
        }
        __syncthreads();
    }
}

}  // namespace ddpk
