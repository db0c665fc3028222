// loss_rows.cu -- what the loss head does around its matrix products, row by row:
// which tokens are learned, their hidden states gathered into rows of the tensor
// cores' layout, the teachers' entries in column order, the statistics joined to
// losses and to the gradients' coefficients, and the hidden states' gradients
// written back to their tokens.
//
// All of it is bound by memory or by latency and small beside the products: with T
// tokens of d elements the gather and the join read and write T d elements each.
// Nothing here uses atomics on values: every sum has one order.
#include <algorithm>
#include <type_traits>

#include "ddp_device.cuh"
#include "loss_internal.h"

namespace ddpk {
namespace {

constexpr int kWarps = kThreads / 32;
constexpr int kMostList = DDP_MAX_TEACHER + 1;

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int d = 16; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
}
template <class T>
__device__ __forceinline__ T warp_sum(T x) {
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// The rank of a row or token number of the group.
__device__ __forceinline__ int rank_of(const LossGroup& g, int row) {
    int i = 0;
    while (i + 1 < g.n && row >= g.row0[i + 1]) ++i;
    return i;
}
// Rows that a product over a rank's rows reads.
__device__ __forceinline__ int padded(int count) { return (count + kTileK - 1) / kTileK * kTileK; }

// Whether a target is a column; one that is neither that nor the ignored value is reported.
__device__ __forceinline__ bool learned(int64_t y, const LossCall& c) {
    if (y == c.ignore_index) return false;
    if (y >= 0 && y < c.vocab) return true;
    report_invalid(c.status);
    return false;
}

// ---- teachers -------------------------------------------------------------------
// A warp a token.  Entries with an index below 0 or a logit of -infinity are none.
__global__ void __launch_bounds__(kThreads) k_teacher(const __grid_constant__ LossGroup g, const __grid_constant__ LossCall c) {
    __shared__ int32_t column[kWarps][kMostList], sorted[kWarps][kMostList];
    __shared__ float share[kWarps][kMostList];
    pdl_release();
    pdl_acquire();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int first = g.row0[0], last = g.row0[g.n];
    for (int at = first + blockIdx.x * kWarps + warp; at < last; at += gridDim.x * kWarps) {
        const int i = rank_of(g, at), t = at - g.row0[i];
        if (t >= g.tokens[i]) continue;
        const int64_t y = g.targets[i] ? g.targets[i][t] : 0;
        bool ok = !g.targets[i] || learned(y, c);      // the same in every lane
        int entries = 0;
        __syncwarp();
        if (ok) {
            const int64_t base = (int64_t)t * c.n_teacher;
            float top = -INFINITY;
            for (int k = lane; k < c.n_teacher; k += 32) {
                const int64_t j = g.indices[i][base + k];
                const float x = c.teacher_dtype == DDP_F32 ? static_cast<const float*>(g.teacher[i])[base + k]
                                                           : bf16_to_f32(static_cast<const uint16_t*>(g.teacher[i])[base + k]);
                if (j >= c.vocab) report_invalid(c.status);
                const bool there = j >= 0 && j < c.vocab && x != -INFINITY;
                column[warp][k] = there ? (int32_t)j : INT32_MAX;
                share[warp][k] = x;
                if (there) top = fmaxf(top, x);
                entries += there;
            }
            entries = warp_sum(entries);
            top = warp_max(top);
            if (top == -INFINITY) top = 0.f;           // NaN entries alone
            float sum = 0.f;
            for (int k = lane; k < c.n_teacher; k += 32)
                if (column[warp][k] != INT32_MAX) sum += expf((share[warp][k] - top) * c.inv_temperature);
            sum = warp_sum(sum);
            float entropy = 0.f;
            for (int k = lane; k < c.n_teacher; k += 32) {
                const float u = (share[warp][k] - top) * c.inv_temperature, q = expf(u) / sum;
                if (column[warp][k] != INT32_MAX && q != 0.f) entropy += q * (u - logf(sum));
                share[warp][k] = q;
            }
            entropy = warp_sum(entropy);
            ok = entries > 0;
            if (lane == 0) {
                c.entropy[at] = entropy;
                if (g.targets[i]) {
                    column[warp][c.n_teacher] = (int32_t)y;
                    share[warp][c.n_teacher] = -1.f;   // the target's mark
                }
            }
        }
        if (lane == 0) c.valid[at] = ok;
        if (!ok) continue;
        __syncwarp();
        // in column order, by counting the entries before each
        for (int k = lane; k < c.list; k += 32) {
            const int32_t mine = column[warp][k];
            int p = 0;
            for (int j = 0; j < c.list; ++j) p += column[warp][j] < mine || (column[warp][j] == mine && j < k);
            sorted[warp][p] = mine;
            c.columns[(int64_t)at * c.list + p] = mine;
            c.share[(int64_t)at * c.list + p] = share[warp][k];
        }
        __syncwarp();
        const int n = entries + (g.targets[i] ? 1 : 0);
        for (int u = lane; u <= c.units; u += 32) {    // entries before the unit
            const int64_t column0 = (int64_t)u * kLossUnit;
            int lo = 0, hi = n;
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (sorted[warp][mid] < column0) lo = mid + 1;
                else hi = mid;
            }
            c.starts[(int64_t)at * (c.units + 1) + u] = (uint16_t)lo;
        }
    }
}

// ---- rows of learned tokens -------------------------------------------------------
// One row to its bf16 planes, zeros from `dim` on; src null: a row of zeros.  A warp.
template <bool F32>
__device__ __forceinline__ void row_to_planes(const void* src, uint16_t* dst, int64_t plane, int dim, int dimp, bool vec,
                                              int lane) {
    for (int x = lane * 8; x < dimp; x += 256) {
        if (F32) {
            float v[8];
            if (src && vec && x + 8 <= dim) {
                const float4 a = ld_stream<float4>(static_cast<const float*>(src) + x);
                const float4 b = ld_stream<float4>(static_cast<const float*>(src) + x + 4);
                v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = src && x + e < dim ? static_cast<const float*>(src)[x + e] : 0.f;
            }
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] = bf16x2_rn(v[2 * e], v[2 * e + 1]);
                    v[2 * e] -= bf16_lo(w[e]);
                    v[2 * e + 1] -= bf16_hi(w[e]);
                }
                *reinterpret_cast<uint4*>(dst + q * plane + x) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else {
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (src && vec && x + 8 <= dim) {
                w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) + x);
            } else if (src) {
                uint32_t h[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = x + e < dim ? static_cast<const uint16_t*>(src)[x + e] : 0;
                w = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
            }
            *reinterpret_cast<uint4*>(dst + x) = w;
        }
    }
}

// Learned tokens' hidden states into rows, in the tokens' order.  A block takes a chunk of a rank's tokens: it counts the
// learned ones before the chunk by itself (8 bytes a token from the L2, for at most kMostChunks blocks a rank: a launch
// of its own for the counts would take longer), places its own, and copies their rows, a warp a row.  A rank's last
// block writes the count and zeroes the rows that pad it.
constexpr int kChunk = 8, kMostChunks = 1024;
__host__ __device__ __forceinline__ int chunk_of(int tokens) {
    const int most = (tokens + kMostChunks - 1) / kMostChunks;
    return most > kChunk ? most : kChunk;
}
__host__ __device__ __forceinline__ int chunks_of(int tokens) {      // one for a rank without tokens: its count
    return tokens > 0 ? (tokens + chunk_of(tokens) - 1) / chunk_of(tokens) : 1;
}

template <bool F32>
__global__ void __launch_bounds__(kThreads) k_gather(const __grid_constant__ LossGroup g, const __grid_constant__ LossCall c,
                                                     int items) {
    __shared__ int32_t sums[kWarps];
    __shared__ int32_t token[kThreads];
    pdl_release();
    pdl_acquire();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (blockIdx.x == 0 && threadIdx.x == 0) *c.done = c.next[0] = c.next[1] = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        int i = 0, chunk = item;
        while (chunk >= chunks_of(g.tokens[i])) chunk -= chunks_of(g.tokens[i++]);
        const int n = g.tokens[i], row0 = g.row0[i], t0 = chunk * chunk_of(n), t1 = min(n, t0 + chunk_of(n));
        const auto is_learned = [&](int t) {
            if (c.alpha != 0.f) return c.valid[row0 + t] != 0;
            const int64_t y = g.targets[i][t];
            return y != c.ignore_index && y >= 0 && y < c.vocab;
        };
        int sum = 0;
#pragma unroll 4
        for (int t = threadIdx.x; t < t0; t += kThreads) sum += is_learned(t);
        sum = warp_sum(sum);
        __syncthreads();
        if (lane == 0) sums[warp] = sum;
        __syncthreads();
        int count = 0;
        for (int k = 0; k < kWarps; ++k) count += sums[k];
        const char* h = static_cast<const char*>(g.hidden[i]);
        const int es = F32 ? 4 : 2;
        const bool vec = ((uintptr_t)h | (uintptr_t)(c.hidden_stride * es)) % 16 == 0;
        uint16_t* rows = static_cast<uint16_t*>(c.gathered) + (int64_t)row0 * c.dimp;
        for (int b = t0; b < t1; b += kThreads) {
            const int t = b + threadIdx.x;
            bool ok = false;
            if (t < t1) ok = c.alpha == 0.f ? learned(g.targets[i][t], c) : is_learned(t);
            const uint32_t there = __ballot_sync(0xffffffffu, ok);
            __syncthreads();
            if (lane == 0) sums[warp] = __popc(there);
            __syncthreads();
            int before = 0, all = 0;
            for (int k = 0; k < kWarps; ++k) {
                if (k < warp) before += sums[k];
                all += sums[k];
            }
            before += __popc(there & ((1u << lane) - 1));
            if (ok) {
                token[before] = t;
                c.row_token[row0 + count + before] = t;
                if (c.alpha == 0.f) c.row_column[row0 + count + before] = (int32_t)g.targets[i][t];
            }
            if (t < t1) {
                c.token_row[row0 + t] = ok ? count + before : -1;
                if (!ok && g.token_losses[i]) g.token_losses[i][t] = 0.f;
            }
            __syncthreads();
            for (int k = warp; k < all; k += kWarps)
                row_to_planes<F32>(h + (int64_t)token[k] * c.hidden_stride * es, rows + (int64_t)(count + k) * c.dimp,
                                   c.rows * c.dimp, c.dim, c.dimp, vec, lane);
            count += all;
        }
        if (t1 == n) {
            if (threadIdx.x == 0) c.counts[g.first + i] = count;
            for (int r = count + warp; r < padded(count); r += kWarps)
                row_to_planes<F32>(nullptr, rows + (int64_t)r * c.dimp, c.rows * c.dimp, c.dim, c.dimp, false, lane);
        }
    }
}

// Matrices [rows][dim] of the group's ranks, each to planes of its own, planes of a rank `bytes` apart.
template <bool F32>
__global__ void __launch_bounds__(kThreads) k_planes(const __grid_constant__ LossWeights m, char* dst, int64_t bytes, int rows,
                                                     int dim, int dimp) {
    pdl_release();
    pdl_acquire();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t stride = (int64_t)dim * (F32 ? 4 : 2);
    for (int64_t at = (int64_t)blockIdx.x * kWarps + warp; at < (int64_t)m.n * rows; at += (int64_t)gridDim.x * kWarps) {
        const int i = (int)(at / rows);
        const int64_t row = at - (int64_t)i * rows;
        const char* src = static_cast<const char*>(m.weights[i]);
        const bool vec = ((uintptr_t)src | (uintptr_t)stride) % 16 == 0;
        row_to_planes<F32>(src + row * stride, reinterpret_cast<uint16_t*>(dst + i * bytes) + row * dimp, (int64_t)rows * dimp, dim,
                           dimp, vec, lane);
    }
}

// ---- losses and coefficients -------------------------------------------------------
// A block takes 32 rows of a rank, a row a lane: each warp joins every 32nd unit's statistics; then a warp a
// row joins the warps' and takes the row's target or list.  The last block adds the blocks' losses.
//
// A sum of exponentials is 1 and the rest, and they stay apart to the end (LossCall::partial): log(1 + rest) of a confident
// row has the rest's digits.  The largest logit stays apart from that logarithm too: a loss is the target's distance from the
// largest logit, 0 where it is that, plus the logarithm.
constexpr int kCombineWarps = 32;
static_assert(kCombineWarps == kLossBlockRows, "a warp a row joins the warps' parts");

template <bool TWO>
__global__ void __launch_bounds__(32 * kCombineWarps, 1) k_combine(const __grid_constant__ LossGroup g,
                                                                   const __grid_constant__ LossCall c, float* loss) {
    using Part = std::conditional_t<TWO, float4, float2>;
    __shared__ float tops[kCombineWarps][33], sums[kCombineWarps][33], sums2[kCombineWarps][33];
    __shared__ float losses[32];
    __shared__ int64_t total;
    __shared__ bool final;
    pdl_release();
    pdl_acquire();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (warp == 0) {
        int64_t n = 0;
        if (c.reduction == DDP_LOSS_WORLD_MEAN)
            for (int i = lane; i < g.world; i += 32) n += c.counts[i];
        n = warp_sum(n);
        if (lane == 0) total = n;
    }
    __syncthreads();
    const float k1 = c.k1, k2 = c.k2;
    const int first = g.row0[0] / kLossBlockRows, last = g.row0[g.n] / kLossBlockRows;
    for (int block = first + blockIdx.x; block < last; block += gridDim.x) {
        const int row = block * kLossBlockRows + lane, i = rank_of(g, block * kLossBlockRows);
        const int count = c.counts[g.first + i], r = row - g.row0[i];
        const bool valid = r < count;
        if (block * kLossBlockRows - g.row0[i] >= count) {
            if (threadIdx.x == 0) c.block_loss[block] = 0.0;
            continue;
        }
        // eight units' loads at a time, none of which waits for another
        float m = -INFINITY, s = 0.f, s2 = 0.f;
        const Part* mine = reinterpret_cast<const Part*>(c.partial) + min(row, (int)c.rows - 1);
        for (int u0 = warp; u0 < c.units; u0 += 8 * kCombineWarps) {
            Part p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = mine[min(u0 + e * kCombineWarps, c.units - 1) * c.rows];
            float top = m;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (u0 + e * kCombineWarps >= c.units) {
                    p[e].x = -INFINITY;
                    p[e].y = 0.f;
                    if constexpr (TWO) p[e].z = 0.f;
                }
                top = fmaxf(top, p[e].x);
            }
            const float ref = top == -INFINITY ? 0.f : top;
            int ones = 0;
            // a sum's rest and its 1 relative to the new reference.  A unit of nothing but -infinity, or none: 0; of those
            // and NaN, which no maximum shows, NaN
            const auto term = [&](float x, float rest, float k) {
                const float scale = exp2f((x - ref) * k);
                return fmaf(rest, scale, x == ref ? 0.f : scale);
            };
            s = term(m, s, k1);
            if constexpr (TWO) s2 = term(m, s2, k2);
            ones += m == ref;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s += term(p[e].x, p[e].y, k1);
                if constexpr (TWO) s2 += term(p[e].x, p[e].z, k2);
                ones += p[e].x == ref;
            }
            s += (float)max(ones - 1, 0);
            if constexpr (TWO) s2 += (float)max(ones - 1, 0);
            m = top;
        }
        tops[warp][lane] = m;
        sums[warp][lane] = s;
        sums2[warp][lane] = s2;
        __syncthreads();
        // a warp a row
        const int rr = block * kLossBlockRows + warp;
        if (rr - g.row0[i] < count) {
            const float part = tops[lane][warp], top = warp_max(part), ref = top == -INFINITY ? 0.f : top;
            const int more = max(__popc(__ballot_sync(0xffffffffu, part == ref)) - 1, 0);
            const auto join = [&](float rest, float k) {
                const float scale = exp2f((part - ref) * k);
                return warp_sum(fmaf(rest, scale, part == ref ? 0.f : scale)) + (float)more;
            };
            const float rest = join(sums[lane][warp], k1), rest2 = TWO ? join(sums2[lane][warp], k2) : rest;
            const bool none = top == -INFINITY;        // no terms at all: no 1 either
            const auto logit = [&](float z) { return fmaf(z - ref, c.cut, z - ref); };     // relative to the largest
            const float log1 = none ? logf(rest) : log1pf(rest), log2 = TWO ? (none ? logf(rest2) : log1pf(rest2)) : log1;
            if (c.value && lane == 0) {
                const float sum = none ? rest : 1.f + rest, sum2 = none ? rest2 : 1.f + rest2;
                float4 coef = make_float4(ref, 1.f / sum, 0.f, 0.f);
                if (TWO) {
                    coef.y = (1.f - c.alpha) / sum;
                    coef.w = c.alpha * c.temperature / sum2;
                } else if (c.alpha != 0.f) {           // alpha 1, or temperature 1
                    coef.y = (1.f - c.alpha + c.alpha * c.temperature) / sum;
                }
                c.coef[rr] = coef;
            }
            if (c.alpha == 0.f) {
                if (lane == 0) {
                    const float d = logit(c.z[rr]) - log1;
                    losses[warp] = -d;
                    if (c.value) c.value[rr] = expm1f(d);
                }
            } else {
                const int64_t token = g.row0[i] + c.row_token[rr], at = token * c.list;
                const int n = c.starts[token * (c.units + 1) + c.units];
                float cross = 0.f, hard = 0.f;
                for (int e = lane; e < n; e += 32) {
                    const float q = c.share[at + e], z = logit(c.z[at + e]);
                    if (q < 0.f) hard += log1 - z;     // the target's entry (its sum is the first: alpha < 1)
                    else if (q != 0.f) cross += q * (log2 - z * c.inv_temperature);
                    if (!c.value) continue;
                    // entries of one column follow each other, and hold one gradient
                    const int32_t column = c.columns[at + e];
                    float shares = 0.f, targets = 0.f;
                    int x = e;
                    while (x > 0 && c.columns[at + x - 1] == column) --x;
                    for (; x < n && c.columns[at + x] == column; ++x) {
                        const float o = c.share[at + x];
                        if (o < 0.f) targets += 1.f;
                        else shares += o;
                    }
                    // e^x - q; where both may be near 1, from e^x - 1
                    const auto less = [](float x, float q) { return x > -0.7f ? expm1f(x) + (1.f - q) : expf(x) - q; };
                    const float soft = c.alpha * c.temperature * less(z * c.inv_temperature - log2, shares);
                    const float label = c.alpha < 1.f ? (1.f - c.alpha) * less(z - log1, targets) : 0.f;
                    c.value[at + e] = soft + label;
                }
                cross = warp_sum(cross);
                hard = warp_sum(hard);
                if (lane == 0) {
                    const float soft = c.alpha * c.temperature * c.temperature * (c.entropy[token] + cross);
                    losses[warp] = c.alpha < 1.f ? (1.f - c.alpha) * hard + soft : soft;
                }
            }
        }
        __syncthreads();
        if (warp == 0) {
            if (valid && g.token_losses[i]) g.token_losses[i][c.row_token[row]] = losses[lane];
            const double sum = warp_sum(valid ? (double)losses[lane] : 0.0);
            if (lane == 0) c.block_loss[block] = sum;
        }
        __syncthreads();
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        final = atomicAdd(c.done, 1) == (int)gridDim.x - 1;
    }
    __syncthreads();
    if (!final) return;
    __threadfence();
    for (int i = warp; i < g.n; i += kCombineWarps) {
        const int count = c.counts[g.first + i];
        double sum = 0.0;
        for (int b = g.row0[i] / kLossBlockRows + lane; b < g.row0[i + 1] / kLossBlockRows; b += 32)
            sum += reinterpret_cast<volatile double*>(c.block_loss)[b];
        sum = warp_sum(sum);
        if (lane == 0) {
            const double f = c.reduction == DDP_LOSS_SUM ? 1.0 : c.reduction == DDP_LOSS_MEAN ? 1.0 / count : (double)g.world / total;
            loss[g.first + i] = count > 0 ? (float)(sum * f) : 0.f;
            if (c.value) c.factor[g.first + i] = count > 0 ? (float)(f * c.scale) : 0.f;
        }
    }
    if (threadIdx.x == 0) *c.done = 0;     // for the next group's launch
}

// ---- kept exponentials to the logits' gradients ---------------------------------------
// dz / f = e 2^(reference - largest) / sum: what the products' own epilogue computes where exponentials are not kept, from 11 bits
// of them for bf16 operands and all for float32.  Of two softmaxes the flatter one's exponentials x are kept; the other's
// are x^r with r <= kKeepPower, which multiplies their rounding, 2^-11 of bf16 operands' ones, by r: up to 2^-9, half of the
// bf16 rounding that follows.  A warp takes kConvertColumns columns of a row.
// Memory bound: 8 x 1024 x 50257 bf16, 1.65 GB read and written, in 0.24 ms by itself (6.8 TB/s), 0.26 between products.
constexpr int kConvertColumns = 1024;

// 2^x and log2 x by the special-function unit where 11 bits were kept, else as exact as they come.
template <bool F32>
__device__ __forceinline__ float power_of_two(float x) {
    if constexpr (F32) return exp2f(x);
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool F32, bool TWO, bool LIST>
__global__ void __launch_bounds__(kThreads) k_convert(const __grid_constant__ LossGroup g, const __grid_constant__ LossCall c,
                                                      const char* kept, uint16_t* piece, int64_t width) {
    constexpr int kSteps = kConvertColumns / 256, kVecs = F32 ? 2 : 1;
    constexpr float kBits = F32 ? 0.f : (float)kKeepBits;
    pdl_release();
    pdl_acquire();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const float k1 = c.k1, k2 = c.k2;
    const bool flat = TWO && k2 < k1;                  // the second softmax's were kept
    const float r = TWO ? (flat ? k1 / k2 : k2 / k1) : 1.f;
    const int64_t parts = (width + kConvertColumns - 1) / kConvertColumns;
    const int64_t rows = g.row0[g.n] - g.row0[0], items = rows * parts;
    for (int64_t item = (int64_t)blockIdx.x * kWarps + warp; item < items; item += (int64_t)gridDim.x * kWarps) {
        const int row = g.row0[0] + (int)(item / parts);
        const int i = rank_of(g, row), t = row - g.row0[i], count = c.counts[g.first + i];
        if (t >= padded(count)) continue;
        const int64_t first = item % parts * kConvertColumns, at = (int64_t)(row - g.row0[0]) * width + first + lane * 8;
        if (t >= count) {
            for (int q = 0; q < (F32 ? 3 : 1); ++q)
#pragma unroll
                for (int j = 0; j < kSteps; ++j)
                    if (first + j * 256 < width)
                        *reinterpret_cast<uint4*>(piece + q * rows * width + at + j * 256) = make_uint4(0u, 0u, 0u, 0u);
            continue;
        }
        uint4 x[kSteps][kVecs];
        float top[kSteps];
#pragma unroll
        for (int j = 0; j < kSteps; ++j)
            if (first + j * 256 < width) {
#pragma unroll
                for (int h = 0; h < kVecs; ++h)
                    x[j][h] = *reinterpret_cast<const uint4*>(kept + (at + j * 256) * (F32 ? 4 : 2) + 16 * h);
                const int64_t u = (first + j * 256 + lane * 8) / kLossUnit;
                top[j] = u < c.units ? c.partial[(u * c.rows + row) * (TWO ? 4 : 2)] : -INFINITY;
            }
        const float4 coef = c.coef[row];
        const int64_t token = LIST ? g.row0[i] + c.row_token[row] : 0;
        const int32_t column = LIST ? 0 : c.row_column[row];
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            if (first + j * 256 >= width) break;
            const int col = (int)first + j * 256 + lane * 8;
            const float ref = top[j] == -INFINITY ? coef.x : top[j];       // of nothing but zeros: any that leaves them so
            float v[8];
            if constexpr (F32) {
                const uint32_t w[8] = {x[j][0].x, x[j][0].y, x[j][0].z, x[j][0].w, x[j][1].x, x[j][1].y, x[j][1].z, x[j][1].w};
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[e]);
            } else {
                const uint32_t w[4] = {x[j][0].x, x[j][0].y, x[j][0].z, x[j][0].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
                    v[2 * e] = f.x;
                    v[2 * e + 1] = f.y;
                }
            }
            const float b1 = (ref - coef.x) * k1, b2 = (ref - coef.x) * k2;
            if (TWO) {
                const float own = flat ? exp2f(b2 - kBits) * coef.w : exp2f(b1 - kBits) * coef.y;
                const float other = (flat ? b1 : b2) - kBits * r, factor = flat ? coef.y : coef.w;
#pragma unroll
                for (int e = 0; e < 8; ++e)            // log2 of 0: -infinity, and 0 again
                    v[e] = fmaf(factor, power_of_two<F32>(fmaf(F32 ? log2f(v[e]) : __log2f(v[e]), r, other)), v[e] * own);
            } else {
                const float own = exp2f(b1 - kBits) * coef.y;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= own;
            }
            // the exact gradient where a target or a teacher has its say
            const auto put = [&](int32_t k, float value) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (k == col + e) v[e] = value;
            };
            if (LIST) {
                if (col < c.vocab) {
                    const uint16_t* starts = c.starts + token * (c.units + 1) + col / kLossUnit;
                    for (int k = starts[0]; k < starts[1]; ++k) {
                        const int32_t there = c.columns[token * c.list + k];
                        if (there >= col && there < col + 8) put(there, c.value[token * c.list + k]);
                    }
                }
            } else if (column >= col && column < col + 8) {
                put(column, c.value[row]);
            }
#pragma unroll
            for (int q = 0; q < (F32 ? 3 : 1); ++q) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] = bf16x2_rn(v[2 * e], v[2 * e + 1]);
                    if (F32) {
                        v[2 * e] -= bf16_lo(w[e]);
                        v[2 * e + 1] -= bf16_hi(w[e]);
                    }
                }
                *reinterpret_cast<uint4*>(piece + q * rows * width + at + j * 256) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

// ---- hidden states' gradients --------------------------------------------------------
// A warp takes 128 * kSteps columns of a token and adds their splits in order.  Few splits come with many tokens: four
// runs of columns at a time then; many splits with few tokens: eight splits' loads at a time (38 splits of 64 tokens by
// 1024, 10 MB: 56 us one split after another, 9 so).
template <bool F32, bool MANY>
__global__ void __launch_bounds__(kThreads) k_join(const __grid_constant__ LossGroup g, const __grid_constant__ LossCall c, int splits,
                                                   int parts) {
    constexpr int kSteps = MANY ? 1 : 4, kSplits = MANY ? 8 : 1;
    pdl_release();
    pdl_acquire();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int first = g.row0[0];
    const int64_t items = (int64_t)(g.row0[g.n] - first) * parts;
    for (int64_t item = (int64_t)blockIdx.x * kWarps + warp; item < items; item += (int64_t)gridDim.x * kWarps) {
        const int at = first + (int)(item / parts), i = rank_of(g, at), t = at - g.row0[i];
        if (t >= g.tokens[i]) continue;
        const int r = c.token_row[at], x0 = (int)(item % parts) * 128 * kSteps + lane * 4;
        char* out = static_cast<char*>(g.grad_hidden[i]) + (int64_t)t * c.dim * (F32 ? 4 : 2);
        const bool vec = ((uintptr_t)g.grad_hidden[i] | (uintptr_t)(c.dim * (F32 ? 4 : 2))) % (F32 ? 16 : 8) == 0;
        float4 v[kSteps] = {};
        const float f = c.factor[g.first + i];
        if (r >= 0 && x0 < c.dim) {
            const float* p = c.acc + ((int64_t)g.row0[i] + r) * c.dimp + x0;
            const int64_t step = c.rows * c.dimp;
            for (int s0 = 0; s0 < splits; s0 += kSplits) {
                float4 q[kSplits][kSteps];
#pragma unroll
                for (int s = 0; s < kSplits; ++s)
#pragma unroll
                    for (int j = 0; j < kSteps; ++j)
                        if (x0 + j * 128 < c.dim) q[s][j] = *reinterpret_cast<const float4*>(p + min(s0 + s, splits - 1) * step + j * 128);
#pragma unroll
                for (int s = 0; s < kSplits; ++s)
#pragma unroll
                    for (int j = 0; j < kSteps; ++j)
                        if (s0 + s < splits && x0 + j * 128 < c.dim)
                            v[j] = make_float4(v[j].x + q[s][j].x, v[j].y + q[s][j].y, v[j].z + q[s][j].z, v[j].w + q[s][j].w);
            }
        }
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            const int x = x0 + j * 128;
            if (x >= c.dim) break;
            const float e[4] = {f * v[j].x, f * v[j].y, f * v[j].z, f * v[j].w};
            if (F32) {
                float* o = reinterpret_cast<float*>(out) + x;
                if (vec) *reinterpret_cast<float4*>(o) = make_float4(e[0], e[1], e[2], e[3]);
                else
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (x + k < c.dim) o[k] = e[k];
            } else {
                uint16_t* o = reinterpret_cast<uint16_t*>(out) + x;
                if (vec) *reinterpret_cast<uint2*>(o) = make_uint2(bf16x2_rn(e[0], e[1]), bf16x2_rn(e[2], e[3]));
                else
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (x + k < c.dim) o[k] = f32_to_bf16_rn(e[k]);
            }
        }
    }
}

// Blocks for `warps` warps' work, four waves at most.
int warp_grid(int64_t warps) { return cap_ctas(std::max<int64_t>(1, std::min<int64_t>((warps + kWarps - 1) / kWarps, 32 * sm_count()))); }

}  // namespace

cudaError_t launch_loss_teacher(const LossGroup& g, const LossCall& c, cudaStream_t stream) {
    return launch_dependent(k_teacher, dim3(warp_grid(g.row0[g.n] - g.row0[0])), dim3(kThreads), 0, stream, g, c);
}

cudaError_t launch_loss_gather(const LossGroup& g, const LossCall& c, cudaStream_t stream) {
    int64_t items = 0;
    for (int i = 0; i < g.n; ++i) items += chunks_of(g.tokens[i]);
    return launch_dependent(c.dtype == DDP_F32 ? k_gather<true> : k_gather<false>, dim3(cap_ctas(items)), dim3(kThreads), 0, stream, g,
                            c, (int)items);
}

cudaError_t launch_loss_planes(const LossWeights& m, void* dst, int64_t bytes, const LossCall& c, cudaStream_t stream) {
    return launch_dependent(c.dtype == DDP_F32 ? k_planes<true> : k_planes<false>, dim3(warp_grid((int64_t)m.n * c.vocab)),
                            dim3(kThreads), 0, stream, m, static_cast<char*>(dst), bytes, c.vocab, c.dim, c.dimp);
}

cudaError_t launch_loss_combine(const LossGroup& g, const LossCall& c, float* loss, cudaStream_t stream) {
    const int64_t blocks = (g.row0[g.n] - g.row0[0]) / kLossBlockRows;
    return launch_dependent(c.two ? k_combine<true> : k_combine<false>, dim3(cap_ctas(std::min<int64_t>(blocks, 2 * sm_count()))),
                            dim3(32 * kCombineWarps), 0, stream, g, c, loss);
}

template <bool F32>
static cudaError_t convert(const LossGroup& g, const LossCall& c, const void* kept, void* piece, int64_t width, cudaStream_t stream) {
    const auto kernel = c.two ? k_convert<F32, true, true> : c.alpha != 0.f ? k_convert<F32, false, true> : k_convert<F32, false, false>;
    const int64_t items = (g.row0[g.n] - g.row0[0]) * ((width + kConvertColumns - 1) / kConvertColumns);
    return launch_dependent(kernel, dim3(warp_grid(items)), dim3(kThreads), 0, stream, g, c, static_cast<const char*>(kept),
                            static_cast<uint16_t*>(piece), width);
}
cudaError_t launch_loss_convert(const LossGroup& g, const LossCall& c, const void* kept, void* piece, int64_t width,
                                cudaStream_t stream) {
    return c.dtype == DDP_F32 ? convert<true>(g, c, kept, piece, width, stream) : convert<false>(g, c, kept, piece, width, stream);
}

cudaError_t launch_loss_join(const LossGroup& g, const LossCall& c, int splits, cudaStream_t stream) {
    const bool many = splits > 4;
    const int parts = (c.dim + (many ? 127 : 511)) / (many ? 128 : 512);
    const auto kernel = c.dtype == DDP_F32 ? (many ? k_join<true, true> : k_join<true, false>)
                                           : (many ? k_join<false, true> : k_join<false, false>);
    return launch_dependent(kernel, dim3(warp_grid((int64_t)(g.row0[g.n] - g.row0[0]) * parts)), dim3(kThreads), 0, stream, g, c,
                            splits, parts);
}

}  // namespace ddpk
