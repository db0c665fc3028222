// adamw.cu -- the AdamW update with gradient clipping in its prologue.
//
// For rank r's tensors, with t = steps[r] + 1 and
// c = min(1, max_norm / (norms[r] + 1e-6)) (1 without norms):
//   g' = c g
//   m <- b1 m + (1 - b1) g'
//   v <- b2 v + (1 - b2) g'^2
//   p <- p - lr wd p - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//   copy <- bf16(p), rounded once, where bf16 weights are kept for the model
// in binary32.  A rank whose norm is not finite is left as it was, its step
// count too.  1 - b^t is -expm1(t ln b): for b near 1 and small t the direct
// difference would lose the bits that the quotient needs.
//
// Clipping costs no pass of its own here: the gradient is in a register.  An
// element moves 28 bytes (fp32: g, p, m, v in, p, m, v out; bf16 gradients with
// bf16 copies the same), so HBM bounds it.
#include <algorithm>
#include <climits>

#include "norm_device.cuh"
#include "optim_internal.h"

namespace ddpk {

constexpr int kAdamVecs = 2;                               // groups of 4 elements a thread takes of a tile
constexpr int64_t kAdamTile = (int64_t)kThreads * 4 * kAdamVecs;   // elements a tile

template <int CAP>
struct AdamWTab {
    int32_t n;
    int32_t tiles;
    float* p[CAP];
    float* m[CAP];
    float* v[CAP];
    const void* g[CAP];
    void* copy[CAP];
    int64_t numel[CAP];
    int32_t tile_end[CAP];     // inclusive prefix of tiles
    int16_t rank[CAP];
    uint8_t lead[CAP];         // elements between the 128-byte boundary before p and p: where tiles are cut
    uint8_t flags[CAP];        // 1: aligned groups of 4 line up in every array, 2: weight decay
};
constexpr int kAdamSmall = 32;
constexpr int kAdamLarge = 560;
static_assert(sizeof(AdamWTab<kAdamLarge>) + 128 <= kMaxParamBytes, "AdamW table exceeds the kernel parameter limit");

static int64_t lead_of(const AdamWItem& it) { return (int64_t)(reinterpret_cast<uintptr_t>(it.p) % 128 / 4); }

int64_t adamw_tiles(const AdamWItem& it, int) { return (lead_of(it) + it.numel + kAdamTile - 1) / kAdamTile; }

struct RankStep {
    float c, step, inv_root;   // clip factor, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
    int32_t skip;
};

__device__ __forceinline__ RankStep rank_step(const AdamWScalars& s, const float* norms, const int32_t* steps, int r) {
    RankStep q{1.f, 0.f, 0.f, 0};
    if (norms) {
        const float norm = norms[r];
        if (!(fabsf(norm) <= 3.402823466e38f)) {
            q.skip = 1;
            return q;
        }
        q.c = fminf(1.f, __fdiv_rn(s.max_norm, norm + 1e-6f));
    }
    const float t = (float)(steps[r] + 1);
    q.step = __fdiv_rn(s.lr, -expm1f(t * s.ln_beta1));
    q.inv_root = __frsqrt_rn(-expm1f(t * s.ln_beta2));
    return q;
}

__device__ __forceinline__ void update(float& p, float& m, float& v, float g, const AdamWScalars& s, const RankStep& q,
                                       float lr_decay) {
    const float gc = g * q.c;
    m = fmaf(s.beta1, m, s.one_minus_beta1 * gc);
    v = fmaf(s.beta2, v, s.one_minus_beta2 * gc * gc);
    const float root = fmaf(__fsqrt_rn(v), q.inv_root, s.eps);
    p -= fmaf(lr_decay, p, q.step * __fdiv_rn(m, root));
}

template <class G> struct GradVec;
template <> struct GradVec<float> {
    float4 w;
    __device__ __forceinline__ void load(const void* g, int64_t e) { w = ld_stream<float4>(static_cast<const float*>(g) + e); }
    __device__ __forceinline__ float at(int l) const { return f32_of(w, l); }
    __device__ static __forceinline__ float one(const void* g, int64_t e) { return static_cast<const float*>(g)[e]; }
};
template <> struct GradVec<uint16_t> {
    uint2 w;
    __device__ __forceinline__ void load(const void* g, int64_t e) { w = ld_stream<uint2>(static_cast<const uint16_t*>(g) + e); }
    __device__ __forceinline__ float at(int l) const {
        const uint32_t h = l < 2 ? w.x : w.y;
        return (l & 1) ? bf16_hi(h) : bf16_lo(h);
    }
    __device__ static __forceinline__ float one(const void* g, int64_t e) { return bf16_to_f32(static_cast<const uint16_t*>(g)[e]); }
};

// One element, through memory.
template <class G, bool COPY, int CAP>
__device__ __forceinline__ void update_one(const AdamWTab<CAP>& b, int i, int64_t e, const AdamWScalars& s,
                                           const RankStep& q, float lr_decay) {
    float p = b.p[i][e], m = b.m[i][e], v = b.v[i][e];
    update(p, m, v, GradVec<G>::one(b.g[i], e), s, q, lr_decay);
    b.p[i][e] = p;
    b.m[i][e] = m;
    b.v[i][e] = v;
    if (COPY) static_cast<uint16_t*>(b.copy[i])[e] = f32_to_bf16_rn(p);
}

template <class G, bool COPY, int CAP>
__global__ void __launch_bounds__(kThreads) k_adamw(const __grid_constant__ AdamWTab<CAP> b, const AdamWScalars s,
                                                    const float* norms, int32_t* steps, int32_t* arrivals, int world,
                                                    int advance) {
    __shared__ RankStep shared_step;
    __shared__ int last;
    pdl_release();
    pdl_acquire();
    for (int tile = blockIdx.x; tile < b.tiles; tile += gridDim.x) {
        const int i = first_past(b.tile_end, b.n, tile);
        const int64_t n = b.numel[i];
        const int64_t e0 = (int64_t)(tile - (i ? b.tile_end[i - 1] : 0)) * kAdamTile - b.lead[i];
        const bool vec = b.flags[i] & 1;
        float4 p[kAdamVecs], m[kAdamVecs], v[kAdamVecs];
        GradVec<G> g[kAdamVecs];
        if (vec) {
#pragma unroll
            for (int u = 0; u < kAdamVecs; ++u) {
                const int64_t e = e0 + 4 * (u * kThreads + (int)threadIdx.x);
                if (e >= 0 && e + 4 <= n) {
                    g[u].load(b.g[i], e);
                    p[u] = ld_stream<float4>(b.p[i] + e);
                    m[u] = ld_stream<float4>(b.m[i] + e);
                    v[u] = ld_stream<float4>(b.v[i] + e);
                }
            }
        }
        if (threadIdx.x == 0) shared_step = rank_step(s, norms, steps, b.rank[i]);     // while the loads are under way
        __syncthreads();
        const RankStep q = shared_step;
        __syncthreads();                         // shared_step is free for the next tile
        if (q.skip) continue;
        const float lr_decay = (b.flags[i] & 2) ? s.lr_decay : 0.f;
        if (vec) {
#pragma unroll
            for (int u = 0; u < kAdamVecs; ++u) {
                const int64_t e = e0 + 4 * (u * kThreads + (int)threadIdx.x);
                if (e >= 0 && e + 4 <= n) {
                    update(p[u].x, m[u].x, v[u].x, g[u].at(0), s, q, lr_decay);
                    update(p[u].y, m[u].y, v[u].y, g[u].at(1), s, q, lr_decay);
                    update(p[u].z, m[u].z, v[u].z, g[u].at(2), s, q, lr_decay);
                    update(p[u].w, m[u].w, v[u].w, g[u].at(3), s, q, lr_decay);
                    st_stream<float4>(b.p[i] + e, p[u]);
                    st_stream<float4>(b.m[i] + e, m[u]);
                    st_stream<float4>(b.v[i] + e, v[u]);
                    if (COPY)
                        st_stream<uint2>(static_cast<uint16_t*>(b.copy[i]) + e,
                                         make_uint2(bf16x2_rn(p[u].x, p[u].y), bf16x2_rn(p[u].z, p[u].w)));
                } else {
                    for (int64_t k = max(e, (int64_t)0); k < min(e + 4, n); ++k) update_one<G, COPY>(b, i, k, s, q, lr_decay);
                }
            }
        } else {
            for (int64_t k = e0 + threadIdx.x; k < e0 + kAdamTile; k += kThreads)
                if (k >= 0 && k < n) update_one<G, COPY>(b, i, k, s, q, lr_decay);
        }
    }
    if (!advance) return;
    // the block that arrives last, when every block has read the counts, advances them
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(arrivals, 1) == (int)gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    if (threadIdx.x == 0) *arrivals = 0;
    for (int r = threadIdx.x; r < world; r += kThreads)
        if (!norms || fabsf(norms[r]) <= 3.402823466e38f) ++steps[r];
}

template <class G, bool COPY, int CAP>
static cudaError_t adamw_cap(const AdamWItem* items, int64_t n, int world, AdamWScalars s, const float* norms,
                             int32_t* steps, int32_t* arrivals, cudaStream_t st) {
    AdamWTab<CAP> b;
    int64_t i = 0;
    do {                                         // a call without elements still counts as a step
        b.n = 0;
        b.tiles = 0;
        for (; i < n && b.n < CAP; ++i, ++b.n) {
            const AdamWItem& it = items[i];
            b.tiles += (int32_t)adamw_tiles(it, 0);
            b.p[b.n] = it.p;
            b.m[b.n] = it.m;
            b.v[b.n] = it.v;
            b.g[b.n] = it.g;
            b.copy[b.n] = it.copy;
            b.numel[b.n] = it.numel;
            b.tile_end[b.n] = b.tiles;
            b.rank[b.n] = (int16_t)it.rank;
            const int64_t lead = lead_of(it);
            const uintptr_t q = (uintptr_t)lead % 4, gs = sizeof(G);
            const bool vec = reinterpret_cast<uintptr_t>(it.m) % 16 == 4 * q &&
                             reinterpret_cast<uintptr_t>(it.v) % 16 == 4 * q &&
                             reinterpret_cast<uintptr_t>(it.g) % (4 * gs) == gs * q &&
                             (!COPY || reinterpret_cast<uintptr_t>(it.copy) % 8 == 2 * q);
            b.lead[b.n] = (uint8_t)lead;
            b.flags[b.n] = (uint8_t)((vec ? 1 : 0) | (it.decay ? 2 : 0));
        }
        const cudaError_t e = launch_dependent(k_adamw<G, COPY, CAP>, dim3(cap_ctas(b.tiles)), dim3(kThreads), 0, st, b,
                                               s, norms, steps, arrivals, world, i >= n ? 1 : 0);
        if (e != cudaSuccess) return e;
    } while (i < n);
    return cudaSuccess;
}

template <class G, bool COPY>
static cudaError_t adamw_n(const AdamWItem* items, int64_t n, int world, AdamWScalars s, const float* norms,
                           int32_t* steps, int32_t* arrivals, cudaStream_t st) {
    if (n <= kAdamSmall) return adamw_cap<G, COPY, kAdamSmall>(items, n, world, s, norms, steps, arrivals, st);
    return adamw_cap<G, COPY, kAdamLarge>(items, n, world, s, norms, steps, arrivals, st);
}

cudaError_t launch_adamw(const AdamWItem* items, int64_t n, int world, int grad_dtype, bool copies, AdamWScalars s,
                         const float* norms, int32_t* steps, int32_t* arrivals, cudaStream_t st) {
    if (grad_dtype == DDP_BF16)
        return copies ? adamw_n<uint16_t, true>(items, n, world, s, norms, steps, arrivals, st)
                      : adamw_n<uint16_t, false>(items, n, world, s, norms, steps, arrivals, st);
    return copies ? adamw_n<float, true>(items, n, world, s, norms, steps, arrivals, st)
                  : adamw_n<float, false>(items, n, world, s, norms, steps, arrivals, st);
}

}  // namespace ddpk
