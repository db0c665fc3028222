// norm_device.cuh -- sums of squares, shared by the kernels that take a norm.
//
// A warp adds the squares of the values its lanes hold in binary32: at most a
// few thousand terms, all positive, so the sum's relative error stays within a
// few units of 2^-24 times the chain length, and far below that on average.
// Everything beyond a warp is added in binary64.  A square leaves binary32's
// range long before its value does (2^-75 squares to nothing, 2^64 to
// infinity), so a warp whose sum falls outside [2^-90, 2^126] squares again in
// binary64, from the registers that still hold the values.  Inside that range
// what underflow took is below 2^-138 a warp, nothing next to 2^-90.
#pragma once

#include "ddp_device.cuh"

namespace ddpk {

// launch_dependent for a kernel whose blocks form clusters of C.
template <int C, class... KArgs, class... Args>
inline cudaError_t launch_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, cudaStream_t st, Args&&... args) {
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
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
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
__device__ __forceinline__ bool in_square_range(float w) { return w >= 0x1p-90f && w <= 0x1p126f; }

// The sum of squares of every value in the warp's U vectors a lane; all lanes
// must call it, all get the sum.  Lanes without data pass zero vectors.
template <class E, int U>
__device__ __forceinline__ double warp_sum_squares(const typename E::V (&x)[U]) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};           // four chains: a quarter of the length, and they overlap
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int l = 0; l < E::L; ++l) {
            const float f = f32_of(x[u], l);
            s[l & 3] = fmaf(f, f, s[l & 3]);
        }
    const float w = warp_sum((s[0] + s[1]) + (s[2] + s[3]));
    if (in_square_range(w)) return (double)w;
    bool some = false;                           // zeros alone need no second pass
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int l = 0; l < E::L; ++l) some |= f32_of(x[u], l) != 0.f;
    if (!__any_sync(0xffffffffu, some)) return 0.0;
    double d = 0.0;
#pragma unroll 1
    for (int u = 0; u < U; ++u) {
        typename E::V v = x[0];
#pragma unroll
        for (int k = 1; k < U; ++k)
            if (k == u) v = x[k];
#pragma unroll
        for (int l = 0; l < E::L; ++l) {
            const double f = (double)f32_of(v, l);
            d = fma(f, f, d);
        }
    }
    return warp_sum(d);
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

// One value a warp -> their sum in thread 0 (undefined elsewhere), added in
// warp order.  `sh` has a slot a warp; the caller puts a barrier between two uses.
__device__ __forceinline__ double block_sum(double warp_total, double* sh) {
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) sh[warp] = warp_total;
    __syncthreads();
    double t = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < warps; ++w) t += sh[w];
    return t;
}

}  // namespace ddpk
