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
constexpr int kAdamMedium = 176;
constexpr int kAdamLarge = 560;
static_assert(sizeof(AdamWTab<kAdamLarge>) + 128 <= kMaxParamBytes, "AdamW table exceeds the kernel parameter limit");

static int64_t lead_of(const AdamWItem& it) { return (int64_t)(reinterpret_cast<uintptr_t>(it.p) % 128 / 4); }

int64_t adamw_tiles(const AdamWItem& it) { return (lead_of(it) + it.numel + kAdamTile - 1) / kAdamTile; }

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

__device__ __forceinline__ void advance_steps(const float* norms, int32_t* steps, int world, int from, int stride) {
    for (int r = from; r < world; r += stride)
        if (!norms || fabsf(norms[r]) <= 3.402823466e38f) ++steps[r];
}

// The counts advance when every block has read them.  In a launch of few
// blocks the one that arrives last does it; a block that arrives waits for its
// stores first, so a launch of many leaves it to a second kernel.
__global__ void __launch_bounds__(kThreads) k_adamw_advance(const float* norms, int32_t* steps, int world) {
    pdl_release();
    pdl_acquire();
    advance_steps(norms, steps, world, threadIdx.x, kThreads);
}

template <class G, bool COPY, int CAP>
__global__ void __launch_bounds__(kThreads) k_adamw(const __grid_constant__ AdamWTab<CAP> b,
                                                    const __grid_constant__ AdamWScalars s, const float* norms,
                                                    int32_t* steps, int32_t* arrivals, int world) {
    __shared__ RankStep shared_step;
    __shared__ int slot;
    pdl_release();
    pdl_acquire();
    for (int tile = blockIdx.x; tile < b.tiles; tile += gridDim.x) {
        const int i = block_first_past(b.tile_end, b.n, tile, &slot);
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
        if (threadIdx.x < 32) {                  // while the loads are under way
            const RankStep q = rank_step(s, norms, steps, b.rank[i]);
            if (threadIdx.x == 0) shared_step = q;
        }
        __syncthreads();
        const RankStep q = shared_step;
        if (tile + (int)gridDim.x < b.tiles) __syncthreads();   // shared_step and slot are free for the next tile
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
    if (!arrivals || threadIdx.x >= 32) return;
    int last = 0;
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(arrivals, 1) == (int)gridDim.x - 1;
    }
    if (!__shfl_sync(0xffffffffu, last, 0)) return;
    __threadfence();
    if (threadIdx.x == 0) *arrivals = 0;
    advance_steps(norms, steps, world, threadIdx.x, 32);
}

constexpr int kAdamArriveTiles = 608;            // a wave of four blocks an SM

struct AdamWPlan {
    std::vector<AdamWTab<kAdamSmall>> small;
    std::vector<AdamWTab<kAdamMedium>> medium;
    std::vector<AdamWTab<kAdamLarge>> large;
};

template <int CAP>
static void fill_tables(const AdamWItem* items, int64_t n, int grad_dtype, bool copies, std::vector<AdamWTab<CAP>>* out) {
    const uintptr_t gs = (uintptr_t)elem_bytes(grad_dtype);
    int64_t i = 0;
    do {                                         // a call without elements still counts as a step
        out->emplace_back();
        AdamWTab<CAP>& b = out->back();
        b.n = 0;
        b.tiles = 0;
        for (; i < n && b.n < CAP; ++i, ++b.n) {
            const AdamWItem& it = items[i];
            b.tiles += (int32_t)adamw_tiles(it);
            b.p[b.n] = it.p;
            b.m[b.n] = it.m;
            b.v[b.n] = it.v;
            b.g[b.n] = it.g;
            b.copy[b.n] = it.copy;
            b.numel[b.n] = it.numel;
            b.tile_end[b.n] = b.tiles;
            b.rank[b.n] = (int16_t)it.rank;
            const int64_t lead = lead_of(it);
            const uintptr_t q = (uintptr_t)lead % 4;
            const bool vec = reinterpret_cast<uintptr_t>(it.m) % 16 == 4 * q &&
                             reinterpret_cast<uintptr_t>(it.v) % 16 == 4 * q &&
                             reinterpret_cast<uintptr_t>(it.g) % (4 * gs) == gs * q &&
                             (!copies || reinterpret_cast<uintptr_t>(it.copy) % 8 == 2 * q);
            b.lead[b.n] = (uint8_t)lead;
            b.flags[b.n] = (uint8_t)((vec ? 1 : 0) | (it.decay ? 2 : 0));
        }
    } while (i < n);
}

std::shared_ptr<const AdamWPlan> make_adamw_plan(const AdamWItem* items, int64_t n, int grad_dtype, bool copies) {
    auto plan = std::make_shared<AdamWPlan>();
    if (n <= kAdamSmall) fill_tables(items, n, grad_dtype, copies, &plan->small);
    else if (n <= kAdamMedium) fill_tables(items, n, grad_dtype, copies, &plan->medium);
    else fill_tables(items, n, grad_dtype, copies, &plan->large);
    return plan;
}

template <class G, bool COPY, int CAP>
static cudaError_t adamw_tables(const std::vector<AdamWTab<CAP>>& tables, int world, const AdamWScalars& s,
                                const float* norms, int32_t* steps, int32_t* arrivals, cudaStream_t st) {
    const bool one = tables.size() == 1 && tables[0].tiles <= kAdamArriveTiles;
    int32_t* const count = one ? arrivals : nullptr;
    for (const AdamWTab<CAP>& b : tables) {
        const cudaError_t e = launch_table(k_adamw<G, COPY, CAP>, dim3(cap_ctas(b.tiles)), dim3(kThreads), st, b, s, norms,
                                           steps, count, world);
        if (e != cudaSuccess) return e;
    }
    return one ? cudaSuccess : launch_table(k_adamw_advance, dim3(1), dim3(kThreads), st, norms, steps, world);
}

template <class G, bool COPY>
static cudaError_t adamw(const AdamWPlan& p, int world, const AdamWScalars& s, const float* norms, int32_t* steps,
                         int32_t* arrivals, cudaStream_t st) {
    if (!p.small.empty()) return adamw_tables<G, COPY>(p.small, world, s, norms, steps, arrivals, st);
    if (!p.medium.empty()) return adamw_tables<G, COPY>(p.medium, world, s, norms, steps, arrivals, st);
    return adamw_tables<G, COPY>(p.large, world, s, norms, steps, arrivals, st);
}

cudaError_t launch_adamw(const AdamWPlan& p, int world, int grad_dtype, bool copies, const AdamWScalars& s,
                         const float* norms, int32_t* steps, int32_t* arrivals, cudaStream_t st) {
    if (grad_dtype == DDP_BF16)
        return copies ? adamw<uint16_t, true>(p, world, s, norms, steps, arrivals, st)
                      : adamw<uint16_t, false>(p, world, s, norms, steps, arrivals, st);
    return copies ? adamw<float, true>(p, world, s, norms, steps, arrivals, st)
                  : adamw<float, false>(p, world, s, norms, steps, arrivals, st);
}

}  // namespace ddpk
