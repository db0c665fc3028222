// loss_small.cu -- the losses and their gradients of little data, in one launch.
//
// A model whose logits are a few thousand needs no tensor cores: what it waits for is
// launches.  A block takes a rank, holds its hidden states, weights and logits in
// shared memory as float32, and does everything the other launches do in order:
// learned tokens, logits, softmax, teacher, losses, both products.  Nothing is
// rounded but the results.  A thread computes kOut outputs of one column of a product, so
// that each weight it reads from shared memory serves kOut sums.  Bound by latency: 16 tokens by 100 x 32 with gradients
// take 10 us replayed from a graph, the launches of the general way 28.
#include <algorithm>

#include "ddp_device.cuh"
#include "loss_internal.h"

namespace ddpk {
namespace {

constexpr int kSmallThreads = 512, kSmallWarps = kSmallThreads / 32;
constexpr int kOut = 4;

template <class T>
__device__ __forceinline__ T all_lanes_sum(T x) {
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}
__device__ __forceinline__ float all_lanes_max(float x) {
#pragma unroll
    for (int d = 16; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
}

template <bool F32>
__device__ __forceinline__ float load(const void* p, int64_t i) {
    return F32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}
template <bool F32>
__device__ __forceinline__ void store(void* p, int64_t i, float x) {
    if (F32) static_cast<float*>(p)[i] = x;
    else static_cast<uint16_t*>(p)[i] = f32_to_bf16_rn(x);
}

// Whether token t of rank i is learned, a warp.  A target or an index that is no column is reported by the rank's own block.
__device__ __forceinline__ bool is_learned(const LossGroup& g, const LossCall& c, int i, int t, int lane, bool report) {
    if (g.targets[i]) {
        const int64_t y = g.targets[i][t];
        if (y == c.ignore_index) return false;
        if (y < 0 || y >= c.vocab) {
            if (report) report_invalid(c.status);
            return false;
        }
    }
    if (c.alpha == 0.f) return true;
    bool any = false;
    for (int k = lane; k < c.n_teacher; k += 32) {
        const int64_t at = (int64_t)t * c.n_teacher + k, j = g.indices[i][at];
        if (report && j >= c.vocab) report_invalid(c.status);
        const float x = c.teacher_dtype == DDP_F32 ? load<true>(g.teacher[i], at) : load<false>(g.teacher[i], at);
        any |= j >= 0 && j < c.vocab && x != -INFINITY;
    }
    return __any_sync(0xffffffffu, any);
}

// Sums over `depth` of a[o * a_out + k * a_step] * b[k * b_step + x] for kOut outputs o, depth k0 .. k1.
__device__ __forceinline__ void dots(float (&sum)[kOut], const float* a, int a_out, int a_step, const float* b, int b_step, int k0,
                                     int k1) {
    for (int k = k0; k < k1; ++k) {
        const float y = b[k * b_step];
#pragma unroll
        for (int o = 0; o < kOut; ++o) sum[o] = fmaf(a[o * a_out + k * a_step], y, sum[o]);
    }
}

template <bool F32>
__global__ void __launch_bounds__(kSmallThreads) k_small(const __grid_constant__ LossGroup g, const __grid_constant__ LossCall c,
                                                         const __grid_constant__ LossSmall m, float* loss) {
    extern __shared__ float shared[];
    __shared__ int64_t total;
    __shared__ int32_t count;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    pdl_release();
    pdl_acquire();
    const int stride = c.dim | 1;                      // odd: a column of rows takes every bank
    const int most = (m.most_tokens + kOut - 1) / kOut * kOut, columns = (c.vocab + kOut - 1) / kOut * kOut;
    float* hs = shared;                                // [most][stride]
    float* ws = hs + most * stride;                    // [vocab][stride]
    float* zs = ws + c.vocab * stride;                 // [most][columns], the logits, then their gradients
    float* losses = zs + most * columns;               // [most]
    float* parts = losses + most;                      // [kSmallThreads * kOut]
    int32_t* learned = reinterpret_cast<int32_t*>(parts + kSmallThreads * kOut);   // [most]
    for (int i = blockIdx.x; i < g.n; i += gridDim.x) {
        const int n = g.tokens[i];
        __syncthreads();
        if (threadIdx.x == 0) {
            count = 0;
            total = 0;
        }
        for (int e = threadIdx.x; e < c.vocab * c.dim; e += kSmallThreads)
            ws[e / c.dim * stride + e % c.dim] = load<F32>(m.weights[i], e);
        for (int t = warp; t < most; t += kSmallWarps) {
            const bool ok = t < n && is_learned(g, c, i, t, lane, true);
            if (lane == 0) learned[t] = ok;
            for (int x = lane; x < c.dim; x += 32)
                hs[t * stride + x] = ok ? load<F32>(g.hidden[i], (int64_t)t * c.hidden_stride + x) : 0.f;
        }
        __syncthreads();
        if (warp == 0) {
            int k = 0;
            for (int t = lane; t < n; t += 32) k += learned[t];
            k = all_lanes_sum(k);
            if (lane == 0) count = k;
        }
        if (c.reduction == DDP_LOSS_WORLD_MEAN) {      // every block counts all ranks' tokens
            int k = 0;
            for (int r = 0; r < g.n; ++r)
                for (int t = warp; t < g.tokens[r]; t += kSmallWarps) k += is_learned(g, c, r, t, lane, false);
            if (lane == 0) atomicAdd(reinterpret_cast<unsigned long long*>(&total), (unsigned long long)k);
        }
        // logits
        for (int e = threadIdx.x; e < most / kOut * c.vocab; e += kSmallThreads) {
            const int t = e / c.vocab * kOut, v = e % c.vocab;
            float sum[kOut] = {};
            dots(sum, hs + t * stride, stride, 1, ws + v * stride, 1, 0, c.dim);
#pragma unroll
            for (int o = 0; o < kOut; ++o) zs[(t + o) * columns + v] = sum[o];
        }
        __syncthreads();
        const double f = c.reduction == DDP_LOSS_SUM    ? 1.0
                         : c.reduction == DDP_LOSS_MEAN ? 1.0 / max(count, 1)
                                                        : (double)g.world / (double)max(total, (int64_t)1);
        const float factor = (float)(f * c.scale);
        // a warp a token: softmaxes, loss, the logits' gradients in the logits' place
        for (int t = warp; t < most; t += kSmallWarps) {
            float* z = zs + t * columns;
            if (!learned[t]) {
                for (int v = lane; v < columns; v += 32) z[v] = 0.f;
                if (lane == 0) {
                    losses[t] = 0.f;
                    if (t < n && g.token_losses[i]) g.token_losses[i][t] = 0.f;
                }
                continue;
            }
            float top = -INFINITY;
            for (int v = lane; v < c.vocab; v += 32) top = fmaxf(top, z[v]);
            top = all_lanes_max(top);
            const float ref = top == -INFINITY ? 0.f : top;
            const bool hard = c.alpha < 1.f, soft = c.alpha != 0.f;
            // the largest terms are ones, counted apart, and the reference stays apart from the sums' logarithms: of a
            // confident token the sum is 1 and little more, and its loss far below a step of its logits
            float s1 = 0.f, s2 = 0.f, ones = 0.f;
            for (int v = lane; v < c.vocab; v += 32) {
                if (z[v] == ref) {
                    ones += 1.f;
                    continue;
                }
                if (hard) s1 += expf(z[v] - ref);
                if (soft) s2 += expf((z[v] - ref) * c.inv_temperature);
            }
            ones = all_lanes_sum(ones);
            s1 = all_lanes_sum(s1);
            s2 = all_lanes_sum(s2);
            const auto log_of = [&](float rest) { return ones == 1.f ? log1pf(rest) : logf(ones + rest); };
            const float log1 = log_of(s1), log2 = log_of(s2);
            const int y = hard ? (int)g.targets[i][t] : 0;
            float result = hard ? (1.f - c.alpha) * ((ref - z[y]) + log1) : 0.f;
            const float a = hard ? (1.f - c.alpha) : 0.f, b = c.alpha * c.temperature;
            const int64_t base = (int64_t)t * c.n_teacher;
            float t_top = -INFINITY, t_sum = 0.f;
            if (soft) {
                for (int k = lane; k < c.n_teacher; k += 32) {
                    const int64_t j = g.indices[i][base + k];
                    const float x = c.teacher_dtype == DDP_F32 ? load<true>(g.teacher[i], base + k) : load<false>(g.teacher[i], base + k);
                    if (j >= 0 && j < c.vocab) t_top = fmaxf(t_top, x);
                }
                t_top = all_lanes_max(t_top);
                if (t_top == -INFINITY) t_top = 0.f;   // NaN entries alone
                for (int k = lane; k < c.n_teacher; k += 32) {
                    const int64_t j = g.indices[i][base + k];
                    const float x = c.teacher_dtype == DDP_F32 ? load<true>(g.teacher[i], base + k) : load<false>(g.teacher[i], base + k);
                    if (j >= 0 && j < c.vocab && x != -INFINITY) t_sum += expf((x - t_top) * c.inv_temperature);
                }
                t_sum = all_lanes_sum(t_sum);
                float kl = 0.f;
                for (int k = lane; k < c.n_teacher; k += 32) {
                    const int64_t j = g.indices[i][base + k];
                    const float x = c.teacher_dtype == DDP_F32 ? load<true>(g.teacher[i], base + k) : load<false>(g.teacher[i], base + k);
                    if (j < 0 || j >= c.vocab || x == -INFINITY) continue;
                    const float u = (x - t_top) * c.inv_temperature, q = expf(u) / t_sum;
                    if (q != 0.f) kl += q * (u - logf(t_sum) + (log2 - (z[j] - ref) * c.inv_temperature));
                }
                result += b * c.temperature * all_lanes_sum(kl);
            }
            if (lane == 0) {
                losses[t] = result;
                if (g.token_losses[i]) g.token_losses[i][t] = result;
            }
            if (!m.grad) continue;
            __syncwarp();
            for (int v = lane; v < c.vocab; v += 32) {
                const float x = z[v] - ref;
                float d = 0.f;
                if (hard) d = a * (v == y ? expm1f(x - log1) : expf(x - log1));
                if (soft) d += b * expf(x * c.inv_temperature - log2);
                z[v] = d;
            }
            __syncwarp();
            if (soft)
                for (int k0 = 0; k0 < c.n_teacher; k0 += 32) {
                    const int k = k0 + lane;
                    const int64_t j = k < c.n_teacher ? g.indices[i][base + k] : -1;
                    const float x = j < 0 ? -INFINITY
                                          : (c.teacher_dtype == DDP_F32 ? load<true>(g.teacher[i], base + k) : load<false>(g.teacher[i], base + k));
                    const bool there = j >= 0 && j < c.vocab && x != -INFINITY;
                    const float q = b * (expf((x - t_top) * c.inv_temperature) / t_sum);
                    // entries of one column one after another, in their order
                    const uint32_t same = __match_any_sync(0xffffffffu, there ? (int)j : -1 - lane);
                    const int turn = __popc(same & ((1u << lane) - 1));
                    for (int e = 0; __any_sync(0xffffffffu, there && turn >= e); ++e) {
                        if (there && turn == e) z[j] -= q;
                        __syncwarp();
                    }
                }
            __syncwarp();
            for (int v = lane; v < columns; v += 32) z[v] = v < c.vocab ? z[v] * factor : 0.f;
        }
        __syncthreads();
        if (warp == 0) {
            double sum = 0.0;
            for (int t = lane; t < n; t += 32) sum += (double)losses[t];
            sum = all_lanes_sum(sum);
            if (lane == 0) loss[g.first + i] = (float)(sum * (count > 0 ? f : 0.0));
        }
        if (!m.grad) continue;
        // hidden states' gradients: kOut tokens of a column a thread, the vocabulary in as many parts as there are threads
        {
            const int tiles = most / kOut * c.dim, split = min(max(kSmallThreads / max(tiles, 1), 1), c.vocab);
            const int depth = (c.vocab + split - 1) / split;
            for (int e0 = 0; e0 < tiles * split; e0 += kSmallThreads) {
                const int e = e0 + threadIdx.x, tile = e % tiles, p = e / tiles;
                const int t = tile / c.dim * kOut, x = tile % c.dim;
                float sum[kOut] = {};
                if (e < tiles * split) dots(sum, zs + t * columns, columns, 1, ws + x, stride, p * depth, min((p + 1) * depth, c.vocab));
                if (split > 1) {                       // one round then
#pragma unroll
                    for (int o = 0; o < kOut; ++o) parts[o * kSmallThreads + threadIdx.x] = sum[o];
                    __syncthreads();
                    if (p == 0)
#pragma unroll
                        for (int o = 0; o < kOut; ++o)
                            for (int q = 1; q < split; ++q) sum[o] += parts[o * kSmallThreads + q * tiles + tile];
                }
                if (e < tiles * split && p == 0)
#pragma unroll
                    for (int o = 0; o < kOut; ++o)
                        if (t + o < n) store<F32>(g.grad_hidden[i], (int64_t)(t + o) * c.dim + x, sum[o]);
            }
        }
        // the weights' gradients: kOut rows of a column a thread
        for (int e = threadIdx.x; e < columns / kOut * c.dim; e += kSmallThreads) {
            const int v = e / c.dim * kOut, x = e % c.dim;
            float sum[kOut] = {};
            dots(sum, zs + v, 1, columns, hs + x, stride, 0, n);
#pragma unroll
            for (int o = 0; o < kOut; ++o) {
                if (v + o >= c.vocab) break;
                const int64_t at = (int64_t)(v + o) * c.dim + x;
                if (m.accumulate) {
                    if (count == 0) continue;
                    sum[o] += load<F32>(m.grads[i], at);
                }
                store<F32>(m.grads[i], at, sum[o]);
            }
        }
    }
}

int64_t small_bytes(const LossGroup& g, const LossCall& c) {
    int64_t n = 1;
    for (int i = 0; i < g.n; ++i) n = std::max<int64_t>(n, g.tokens[i]);
    n = (n + kOut - 1) / kOut * kOut;
    const int64_t stride = c.dim | 1, columns = (c.vocab + kOut - 1) / kOut * kOut;
    return 4 * ((n + c.vocab) * stride + n * columns + 2 * n + kSmallThreads * kOut);
}

}  // namespace

bool loss_is_small(const LossGroup& g, const LossCall& c) {
    int64_t n = 1, entries = 0;
    for (int i = 0; i < g.n; ++i) {
        n = std::max<int64_t>(n, g.tokens[i]);
        entries += (int64_t)g.tokens[i] * c.n_teacher;
    }
    return g.n == g.world && (int64_t)c.vocab * c.dim <= kSmallWeights && n * c.vocab * c.dim <= kSmallWork &&
           entries <= kSmallEntries && small_bytes(g, c) <= 200 * 1024;
}

cudaError_t launch_loss_small(const LossGroup& g, const LossCall& c, LossSmall m, float* loss, cudaStream_t stream) {
    m.most_tokens = 1;
    for (int i = 0; i < g.n; ++i) m.most_tokens = std::max(m.most_tokens, g.tokens[i]);
    const auto kernel = c.dtype == DDP_F32 ? k_small<true> : k_small<false>;
    const int bytes = (int)small_bytes(g, c);
    const cudaError_t e = allow_shared_memory((const void*)kernel, 200 * 1024);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(cap_ctas(g.n)), dim3(kSmallThreads), bytes, stream, g, c, m, loss);
}

}  // namespace ddpk
