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
// bf16 copies the same), so HBM bounds it: 7.18 TB/s on 2 ranks x 355M fp32.
// A thread keeps two groups of four elements of every array in flight, three
// blocks an SM (one group up to 4M elements and for fp32 gradients with
// copies, four or five blocks), and one warp works out the rank's scalars while
// they are.  Where one array lies differently against its 16 or 8 bytes all go
// element by element: 25.6M elements with gradients packed at odd offsets and
// the rest apart 169 us in fp32 (4.23 TB/s; lined up 106), 171 with bf16
// gradients and copies (108), 157 with fp32 gradients and copies (122).
// Nothing of a block waits for its stores: what each costs is measured at
// make_adamw_plan and k_adamw_advance.
#include <algorithm>
#include <climits>

#include "norm_device.cuh"
#include "optim_internal.h"

namespace ddpk {

// Elements of a tile in which a thread takes `vecs` groups of 4.
constexpr int64_t adamw_tile(int vecs) { return (int64_t)kThreads * 4 * vecs; }

struct Item {                  // side by side: a block finds one line of a cold constant cache, not one a field
    float* p;
    float* m;
    float* v;
    const void* g;
    void* copy;
    int64_t numel;
    int32_t first;             // its first tile
    int16_t rank;
    uint8_t lead;              // elements between the 128-byte boundary before p and p: where tiles are cut
    uint8_t flags;             // 1: aligned groups of 4 line up in every array, 2: weight decay
};
static_assert(sizeof(Item) == kAdamWEntry, "the workspace counts on it");

template <int CAP>
struct AdamWTab {
    static constexpr bool kDevice = false;
    int32_t n;
    int32_t tiles;
    int32_t tile_end[CAP];     // inclusive prefix of tiles
    Item item[CAP];
};
struct AdamWDev {              // the same in device memory
    static constexpr bool kDevice = true;
    int32_t n, tiles;
    const int32_t* tile_end;
    const Item* item;
};
constexpr int kAdamSmall = 32;
constexpr int kAdamMedium = 176;
constexpr int kAdamLarge = 536;
static_assert(sizeof(AdamWTab<kAdamLarge>) + 128 <= kMaxParamBytes, "AdamW table exceeds the kernel parameter limit");

static int64_t lead_of(const AdamWItem& it) { return (int64_t)(reinterpret_cast<uintptr_t>(it.p) % 128 / 4); }

static int64_t adamw_tiles(const AdamWItem& it, int64_t tile) { return (lead_of(it) + it.numel + tile - 1) / tile; }
int64_t adamw_tiles(const AdamWItem& it) { return adamw_tiles(it, adamw_tile(1)); }

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
template <class G, bool COPY, class TAB>
__device__ __forceinline__ void update_one(const TAB& b, int i, int64_t e, const AdamWScalars& s,
                                           const RankStep& q, float lr_decay) {
    float p = b.item[i].p[e], m = b.item[i].m[e], v = b.item[i].v[e];
    update(p, m, v, GradVec<G>::one(b.item[i].g, e), s, q, lr_decay);
    b.item[i].p[e] = p;
    b.item[i].m[e] = m;
    b.item[i].v[e] = v;
    if (COPY) static_cast<uint16_t*>(b.item[i].copy)[e] = f32_to_bf16_rn(p);
}

__device__ __forceinline__ void advance_steps(const float* norms, int32_t* steps, int world, int from, int stride) {
    for (int r = from; r < world; r += stride)
        if (!norms || fabsf(norms[r]) <= 3.402823466e38f) ++steps[r];
}

// The counts advance when every block has read them.  In a launch of few
// blocks the one that arrives last does it; a block that arrives waits for its
// stores first, so a launch of many leaves it to a second kernel (2 ranks x 355M
// fp32: 2.77 against 3.19 ms).
__global__ void __launch_bounds__(kThreads) k_adamw_advance(const float* norms, int32_t* steps, int world) {
    pdl_release();
    pdl_acquire();
    advance_steps(norms, steps, world, threadIdx.x, kThreads);
}

// fp32 gradients with copies never take two groups a thread (make_adamw_plan):
// no such kernel is built.
template <class G, bool COPY>
constexpr bool kOneGroup = COPY && sizeof(G) == 4;

// V: groups of 4 elements a thread takes.
template <class G, bool COPY, int V, class TAB>
__global__ void __launch_bounds__(kThreads, V == 2 ? 3 : kOneGroup<G, COPY> ? 5 : 4) k_adamw(const __grid_constant__ TAB b,
                                                    const __grid_constant__ AdamWScalars s, const float* norms,
                                                    int32_t* steps, int32_t* arrivals, int world) {
    static_assert(V == 1 || !kOneGroup<G, COPY>, "no call reaches this kernel");
    constexpr int64_t kTile = adamw_tile(V);
    __shared__ RankStep shared_step;
    __shared__ int slot;
    AcquireOnce acquire;
    pdl_release();
    if constexpr (TAB::kDevice) acquire();
    for (int tile = blockIdx.x; tile < b.tiles; tile += gridDim.x) {
        const int i = block_first_past(b.tile_end, b.n, tile, &slot);
        const int64_t n = b.item[i].numel;
        const int64_t e0 = (int64_t)(tile - b.item[i].first) * kTile - b.item[i].lead;
        const bool vec = b.item[i].flags & 1;
        acquire();
        float4 p[V], m[V], v[V];
        GradVec<G> g[V];
        if (vec) {
#pragma unroll
            for (int u = 0; u < V; ++u) {
                const int64_t e = e0 + 4 * (u * kThreads + (int)threadIdx.x);
                if (e >= 0 && e + 4 <= n) {
                    g[u].load(b.item[i].g, e);
                    p[u] = ld_stream<float4>(b.item[i].p + e);
                    m[u] = ld_stream<float4>(b.item[i].m + e);
                    v[u] = ld_stream<float4>(b.item[i].v + e);
                }
            }
        }
        if (threadIdx.x < 32) {                  // while the loads are under way
            const RankStep q = rank_step(s, norms, steps, b.item[i].rank);
            if (threadIdx.x == 0) shared_step = q;
        }
        __syncthreads();
        const RankStep q = shared_step;
        if (tile + (int)gridDim.x < b.tiles) __syncthreads();   // shared_step and slot are free for the next tile
        if (q.skip) continue;
        const float lr_decay = (b.item[i].flags & 2) ? s.lr_decay : 0.f;
        if (vec) {
#pragma unroll
            for (int u = 0; u < V; ++u) {
                const int64_t e = e0 + 4 * (u * kThreads + (int)threadIdx.x);
                if (e >= 0 && e + 4 <= n) {
                    update(p[u].x, m[u].x, v[u].x, g[u].at(0), s, q, lr_decay);
                    update(p[u].y, m[u].y, v[u].y, g[u].at(1), s, q, lr_decay);
                    update(p[u].z, m[u].z, v[u].z, g[u].at(2), s, q, lr_decay);
                    update(p[u].w, m[u].w, v[u].w, g[u].at(3), s, q, lr_decay);
                    st_stream<float4>(b.item[i].p + e, p[u]);
                    st_stream<float4>(b.item[i].m + e, m[u]);
                    st_stream<float4>(b.item[i].v + e, v[u]);
                    if (COPY)
                        st_stream<uint2>(static_cast<uint16_t*>(b.item[i].copy) + e,
                                         make_uint2(bf16x2_rn(p[u].x, p[u].y), bf16x2_rn(p[u].z, p[u].w)));
                } else {
                    for (int64_t k = max(e, (int64_t)0); k < min(e + 4, n); ++k) update_one<G, COPY>(b, i, k, s, q, lr_decay);
                }
            }
        } else {
            for (int64_t k = e0 + threadIdx.x; k < e0 + kTile; k += kThreads)
                if (k >= 0 && k < n) update_one<G, COPY>(b, i, k, s, q, lr_decay);
        }
    }
    acquire();
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
constexpr int64_t kAdamSpread = 4 << 20;         // elements

struct AdamWPlan {
    int vecs = 2;
    std::vector<AdamWTab<kAdamSmall>> small;
    std::vector<AdamWTab<kAdamMedium>> medium;
    std::vector<AdamWTab<kAdamLarge>> large;
    DeviceTable device;                          // more items than one launch's table takes, for little data
    AdamWDev dev{};                              // with offsets for addresses
};

const DeviceTable* adamw_plan_table(const AdamWPlan& plan) { return plan.device.image.empty() ? nullptr : &plan.device; }

static Item item_of(const AdamWItem& it, int32_t first, int grad_dtype, bool copies) {
    const uintptr_t gs = (uintptr_t)elem_bytes(grad_dtype);
    const int64_t lead = lead_of(it);
    const uintptr_t q = (uintptr_t)lead % 4;
    const bool vec = reinterpret_cast<uintptr_t>(it.m) % 16 == 4 * q && reinterpret_cast<uintptr_t>(it.v) % 16 == 4 * q &&
                     reinterpret_cast<uintptr_t>(it.g) % (4 * gs) == gs * q &&
                     (!copies || reinterpret_cast<uintptr_t>(it.copy) % 8 == 2 * q);
    return Item{it.p, it.m, it.v, it.g, it.copy, it.numel, first, (int16_t)it.rank, (uint8_t)lead,
                (uint8_t)((vec ? 1 : 0) | (it.decay ? 2 : 0))};
}

// Items [i, n) as far as `most` goes into one table; returns where it stopped.
template <class Ends, class Entries>
static int64_t fill_table(const AdamWItem* items, int64_t i, int64_t n, int64_t most, int64_t tile, int grad_dtype,
                          bool copies, Ends ends, Entries entries, int32_t* count, int32_t* tiles) {
    *count = 0;
    *tiles = 0;
    for (; i < n && *count < most; ++i, ++*count) {
        entries[*count] = item_of(items[i], *tiles, grad_dtype, copies);
        *tiles += (int32_t)adamw_tiles(items[i], tile);
        ends[*count] = *tiles;
    }
    return i;
}

template <int CAP>
static void fill_tables(const AdamWItem* items, int64_t n, int64_t tile, int grad_dtype, bool copies,
                        std::vector<AdamWTab<CAP>>* out) {
    int64_t i = 0;
    do {                                         // a call without elements still counts as a step
        out->emplace_back();
        AdamWTab<CAP>& b = out->back();
        i = fill_table(items, i, n, CAP, tile, grad_dtype, copies, b.tile_end, b.item, &b.n, &b.tiles);
    } while (i < n);
}

std::shared_ptr<const AdamWPlan> make_adamw_plan(const AdamWItem* items, int64_t n, int grad_dtype, bool copies) {
    auto plan = std::make_shared<AdamWPlan>();
    // two groups a thread keep more loads in flight, one spreads a small call
    // over the SMs: 1M fp32 elements 7.3 against 9.6 us, 25.5M 111 against 105.
    // fp32 gradients with copies, seven streams of four bytes and one of two,
    // take one in five blocks an SM: 355M 1514 against 1636 us (bf16 gradients
    // 1413 against 1396, fp32 without copies 1422 against 1376)
    int64_t numel = 0;
    for (int64_t i = 0; i < n; ++i) numel += items[i].numel;
    plan->vecs = numel <= kAdamSpread || (copies && grad_dtype == DDP_F32) ? 1 : 2;
    const int64_t tile = adamw_tile(plan->vecs);
    if (n <= kAdamSmall) fill_tables(items, n, tile, grad_dtype, copies, &plan->small);
    else if (n <= kAdamMedium) fill_tables(items, n, tile, grad_dtype, copies, &plan->medium);
    else if (table_on_device((n + kAdamLarge - 1) / kAdamLarge, numel * (24 + elem_bytes(grad_dtype) + (copies ? 2 : 0)))) {
        DeviceTable& t = plan->device;
        t.entries_at = (4 * n + 15) / 16 * 16;
        t.image.assign((size_t)(t.entries_at + (n * kAdamWEntry + 15) / 16 * 16), 0);
        fill_table(items, 0, n, n, tile, grad_dtype, copies, reinterpret_cast<int32_t*>(t.image.data()),
                   reinterpret_cast<Item*>(t.image.data() + t.entries_at), &plan->dev.n, &plan->dev.tiles);
    } else fill_tables(items, n, tile, grad_dtype, copies, &plan->large);
    return plan;
}

template <class G, bool COPY, int V, class TAB>
static cudaError_t adamw_table(const TAB& b, int world, const AdamWScalars& s, const float* norms, int32_t* steps,
                               int32_t* arrivals, cudaStream_t st) {
    return launch_table(k_adamw<G, COPY, V, TAB>, dim3(cap_ctas(b.tiles)), dim3(kThreads), st, b, s, norms, steps, arrivals,
                        world);
}

// `one` launch of few tiles advances the counts itself.
template <class G, bool COPY, int V, class TAB>
static cudaError_t adamw_tables(const TAB* tables, size_t n, int world, const AdamWScalars& s, const float* norms,
                                int32_t* steps, int32_t* arrivals, cudaStream_t st) {
    const bool one = n == 1 && tables[0].tiles <= kAdamArriveTiles;
    int32_t* const count = one ? arrivals : nullptr;
    for (size_t k = 0; k < n; ++k) {
        const cudaError_t e = adamw_table<G, COPY, V>(tables[k], world, s, norms, steps, count, st);
        if (e != cudaSuccess) return e;
    }
    return one ? cudaSuccess : launch_table(k_adamw_advance, dim3(1), dim3(kThreads), st, norms, steps, world);
}

template <class G, bool COPY, int V>
static cudaError_t adamw_size(const AdamWPlan& p, const char* table, int world, const AdamWScalars& s, const float* norms,
                              int32_t* steps, int32_t* arrivals, cudaStream_t st) {
    auto run = [&](const auto& t) {
        return adamw_tables<G, COPY, V>(t.data(), t.size(), world, s, norms, steps, arrivals, st);
    };
    if (!p.small.empty()) return run(p.small);
    if (!p.medium.empty()) return run(p.medium);
    if (!p.large.empty()) return run(p.large);
    AdamWDev d = p.dev;
    d.tile_end = reinterpret_cast<const int32_t*>(table);
    d.item = reinterpret_cast<const Item*>(table + p.device.entries_at);
    return adamw_tables<G, COPY, V>(&d, 1, world, s, norms, steps, arrivals, st);
}

template <class G, bool COPY>
static cudaError_t adamw(const AdamWPlan& p, const char* table, int world, const AdamWScalars& s, const float* norms,
                         int32_t* steps, int32_t* arrivals, cudaStream_t st) {
    if constexpr (!kOneGroup<G, COPY>)
        if (p.vecs == 2) return adamw_size<G, COPY, 2>(p, table, world, s, norms, steps, arrivals, st);
    return adamw_size<G, COPY, 1>(p, table, world, s, norms, steps, arrivals, st);
}

cudaError_t launch_adamw(const AdamWPlan& p, const char* table, int world, int grad_dtype, bool copies,
                         const AdamWScalars& s, const float* norms, int32_t* steps, int32_t* arrivals, cudaStream_t st) {
    if (grad_dtype == DDP_BF16)
        return copies ? adamw<uint16_t, true>(p, table, world, s, norms, steps, arrivals, st)
                      : adamw<uint16_t, false>(p, table, world, s, norms, steps, arrivals, st);
    return copies ? adamw<float, true>(p, table, world, s, norms, steps, arrivals, st)
                  : adamw<float, false>(p, table, world, s, norms, steps, arrivals, st);
}

}  // namespace ddpk
