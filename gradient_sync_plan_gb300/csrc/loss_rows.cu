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
#include <cfloat>

#include "ddp_device.cuh"
#include "loss_internal.h"

namespace ddpk {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kScanThreads = 1024;
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
    atomicExch(c.status, DDP_ERR_INVALID);
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
                if (j >= c.vocab) atomicExch(c.status, DDP_ERR_INVALID);
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
// A block a rank; four tokens a thread and pass.
__global__ void __launch_bounds__(kScanThreads) k_scan(const __grid_constant__ LossGroup g, const __grid_constant__ LossCall c) {
    __shared__ int32_t before[kScanThreads / 32];
    pdl_release();
    pdl_acquire();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (blockIdx.x == 0 && threadIdx.x == 0) *c.done = c.next[0] = c.next[1] = 0;
    for (int i = blockIdx.x; i < g.n; i += gridDim.x) {
        const int row0 = g.row0[i], n = g.tokens[i];
        int count = 0;
        for (int t0 = 0; t0 < n; t0 += 4 * kScanThreads) {
            const int mine = t0 + 4 * threadIdx.x;
            int64_t y[4];
            bool ok[4];
            int sum = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = mine + e < n && g.targets[i] ? g.targets[i][mine + e] : 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                ok[e] = mine + e < n && (c.alpha == 0.f ? learned(y[e], c) : c.valid[row0 + mine + e] != 0);
                sum += ok[e];
            }
            int in_warp = sum;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, in_warp, d);
                if (lane >= d) in_warp += x;
            }
            if (lane == 31) before[warp] = in_warp;
            __syncthreads();
            int row = count + in_warp - sum;
            for (int k = 0; k < kScanThreads / 32; ++k) {
                if (k < warp) row += before[k];
                count += before[k];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = mine + e;
                if (t >= n) break;
                c.token_row[row0 + t] = ok[e] ? row : -1;
                if (ok[e]) {
                    c.row_token[row0 + row] = t;
                    c.row_column[row0 + row] = (int32_t)y[e];
                    ++row;
                } else if (g.token_losses[i]) {
                    g.token_losses[i][t] = 0.f;
                }
            }
            __syncthreads();
        }
        if (threadIdx.x == 0) c.counts[g.first + i] = count;
    }
}

// One row to its bf16 planes, zeros from `dim` on; src null: a row of zeros.  A warp.
template <bool F32>
__device__ __forceinline__ void row_to_planes(const void* src, uint16_t* dst, int64_t plane, int dim, int dimp, bool vec,
                                              int lane) {
    for (int x = lane * 8; x < dimp; x += 256) {
        if (F32) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = src && x + e < dim ? static_cast<const float*>(src)[x + e] : 0.f;
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

template <bool F32>
__global__ void __launch_bounds__(kThreads) k_gather(const __grid_constant__ LossGroup g, const __grid_constant__ LossCall c) {
    pdl_release();
    pdl_acquire();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int first = g.row0[0], last = g.row0[g.n];
    for (int row = first + blockIdx.x * kWarps + warp; row < last; row += gridDim.x * kWarps) {
        const int i = rank_of(g, row), r = row - g.row0[i], count = c.counts[g.first + i];
        if (r >= padded(count)) continue;
        const char* h = static_cast<const char*>(g.hidden[i]);
        const int es = F32 ? 4 : 2;
        const bool vec = ((uintptr_t)h | (uintptr_t)(c.hidden_stride * es)) % 16 == 0;
        const void* src = r < count ? h + (int64_t)c.row_token[row] * c.hidden_stride * es : nullptr;
        row_to_planes<F32>(src, static_cast<uint16_t*>(c.gathered) + (int64_t)row * c.dimp, c.rows * c.dimp, c.dim, c.dimp, vec,
                           lane);
    }
}

template <bool F32>
__global__ void __launch_bounds__(kThreads) k_planes(const char* src, uint16_t* dst, int64_t rows, int dim, int dimp) {
    pdl_release();
    pdl_acquire();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t stride = (int64_t)dim * (F32 ? 4 : 2);
    const bool vec = ((uintptr_t)src | (uintptr_t)stride) % 16 == 0;
    for (int64_t row = (int64_t)blockIdx.x * kWarps + warp; row < rows; row += (int64_t)gridDim.x * kWarps)
        row_to_planes<F32>(src + row * stride, dst + row * dimp, rows * dimp, dim, dimp, vec, lane);
}

// ---- losses and coefficients -------------------------------------------------------
// A block takes 32 rows of a rank, a row a lane: each warp joins every 32nd unit's statistics, the first joins the
// warps'.  Distillation then takes the rows' lists, a warp a row.  The last block adds the blocks' losses.
constexpr int kCombineWarps = 32;
__device__ __forceinline__ void join_stats(float& m, float& s, float& s2, float om, float os, float os2, float k1, float k2) {
    const float top = fmaxf(m, om);
    const float ref = top == -INFINITY ? 0.f : top;
    const float a = m - ref, b = om - ref;
    s = s * exp2f(a * k1) + os * exp2f(b * k1);
    s2 = s2 * exp2f(a * k2) + os2 * exp2f(b * k2);
    m = top;
}

template <bool TWO>
__global__ void __launch_bounds__(32 * kCombineWarps) k_combine(const __grid_constant__ LossGroup g, const __grid_constant__ LossCall c,
                                                      float* loss) {
    __shared__ float tops[kCombineWarps][32], sums[kCombineWarps][32], sums2[kCombineWarps][32];
    __shared__ float lse1[32], lse2[32], losses[32];
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
    const float k1 = TWO ? kLog2e : c.inv_temperature * kLog2e, k2 = c.inv_temperature * kLog2e;
    const int first = g.row0[0] / kLossBlockRows, last = g.row0[g.n] / kLossBlockRows;
    for (int block = first + blockIdx.x; block < last; block += gridDim.x) {
        const int row = block * kLossBlockRows + lane, i = rank_of(g, block * kLossBlockRows);
        const int count = c.counts[g.first + i], r = row - g.row0[i];
        const bool valid = r < count;
        if (block * kLossBlockRows - g.row0[i] >= count) {
            if (threadIdx.x == 0) c.block_loss[block] = 0.0;
            continue;
        }
        // a warp's maximum first, so that the loads of each pass do not wait for one another
        float m = -INFINITY, s = 0.f, s2 = 0.f;
        const int step = TWO ? 4 : 2;
        if (valid) {
#pragma unroll 8
            for (int u = warp; u < c.units; u += kCombineWarps) m = fmaxf(m, c.partial[((int64_t)u * c.rows + row) * step]);
            const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll 8
            for (int u = warp; u < c.units; u += kCombineWarps) {
                const int64_t at = (int64_t)u * c.rows + row;
                if (TWO) {
                    const float4 p = reinterpret_cast<const float4*>(c.partial)[at];
                    s += p.y * exp2f((p.x - ref) * k1);
                    s2 += p.z * exp2f((p.x - ref) * k2);
                } else {
                    const float2 p = reinterpret_cast<const float2*>(c.partial)[at];
                    s += p.y * exp2f((p.x - ref) * k1);
                }
            }
        }
        tops[warp][lane] = m;
        sums[warp][lane] = s;
        sums2[warp][lane] = s2;
        __syncthreads();
        const double f = c.reduction == DDP_LOSS_SUM ? 1.0 : c.reduction == DDP_LOSS_MEAN ? 1.0 / count : (double)g.world / total;
        const float factor = (float)(f * c.scale);
        if (warp == 0 && valid) {
            for (int k = 1; k < kCombineWarps; ++k) join_stats(m, s, s2, tops[k][lane], sums[k][lane], sums2[k][lane], k1, k2);
            const float single = TWO ? 1.f : c.inv_temperature;
            lse1[lane] = m * single + logf(s);
            lse2[lane] = TWO ? m * c.inv_temperature + logf(s2) : lse1[lane];
            if (c.value) {
                float4 coef = make_float4(lse1[lane] * kLog2e, factor, 0.f, 0.f);
                if (TWO) {
                    coef.y = (1.f - c.alpha) * factor;
                    coef.z = lse2[lane] * kLog2e;
                    coef.w = c.alpha * c.temperature * factor;
                } else if (c.alpha != 0.f) {           // alpha 1, or temperature 1
                    coef.y = (1.f - c.alpha + c.alpha * c.temperature) * factor;
                }
                c.coef[row] = coef;
            }
            if (c.alpha == 0.f) {
                const float d = c.z[row] - lse1[lane];
                losses[lane] = -d;
                if (c.value) c.value[row] = factor * expm1f(d);
            }
        }
        if (c.alpha != 0.f) {
            __syncthreads();
            for (int k = warp; k < kLossBlockRows; k += kCombineWarps) {
                const int rr = block * kLossBlockRows + k;
                if (rr - g.row0[i] >= count) break;
                const int64_t token = g.row0[i] + c.row_token[rr], at = token * c.list;
                const int n = c.starts[token * (c.units + 1) + c.units];
                const float a = lse1[k], b = lse2[k];
                float cross = 0.f, hard = 0.f;
                for (int e = lane; e < n; e += 32) {
                    const float q = c.share[at + e], z = c.z[at + e];
                    if (q < 0.f) hard += a - z;        // the target's entry (its lse is the first: alpha < 1)
                    else if (q != 0.f) cross += q * (b - z * c.inv_temperature);
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
                    const float soft = c.alpha * c.temperature * (expf(z * c.inv_temperature - b) - shares);
                    const float label = c.alpha < 1.f ? (1.f - c.alpha) * (expf(z - a) - targets) : 0.f;
                    c.value[at + e] = factor * (soft + label);
                }
                cross = warp_sum(cross);
                hard = warp_sum(hard);
                if (lane == 0) {
                    const float soft = c.alpha * c.temperature * c.temperature * (c.entropy[token] + cross);
                    losses[k] = c.alpha < 1.f ? (1.f - c.alpha) * hard + soft : soft;
                }
            }
            __syncthreads();
        }
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
        }
    }
    if (threadIdx.x == 0) *c.done = 0;     // for the next group's launch
}

// ---- kept exponentials to the logits' gradients ---------------------------------------
// dz = f e 2^(reference - lse): what the products' own epilogue computes where exponentials are not kept, rounded to
// bf16 once more from 11 bits.  Of two softmaxes the flatter one's exponentials x are kept; the other's are x^r with
// r <= kKeepPower, which multiplies their rounding by r.  A warp takes kConvertColumns columns of a row; memory bound.
constexpr int kConvertColumns = 1024;

template <bool TWO, bool LIST>
__global__ void __launch_bounds__(kThreads) k_convert(const __grid_constant__ LossGroup g, const __grid_constant__ LossCall c,
                                                      uint16_t* piece, int64_t width) {
    pdl_release();
    pdl_acquire();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const float k1 = TWO ? kLog2e : c.inv_temperature * kLog2e, k2 = c.inv_temperature * kLog2e, kept = TWO ? fminf(k1, k2) : k1;
    const float r1 = k1 / kept, r2 = k2 / kept;
    const int64_t parts = (width + kConvertColumns - 1) / kConvertColumns;
    const int64_t items = (g.row0[g.n] - g.row0[0]) * parts;
    for (int64_t item = (int64_t)blockIdx.x * kWarps + warp; item < items; item += (int64_t)gridDim.x * kWarps) {
        const int row = g.row0[0] + (int)(item / parts);
        const int i = rank_of(g, row), r = row - g.row0[i], count = c.counts[g.first + i];
        if (r >= padded(count)) continue;
        const int64_t first = item % parts * kConvertColumns;
        uint16_t* at = piece + (int64_t)(row - g.row0[0]) * width + first + lane * 8;
        if (r >= count) {
#pragma unroll
            for (int j = 0; j < kConvertColumns / 256; ++j)
                if (first + j * 256 < width) *reinterpret_cast<uint4*>(at + j * 256) = make_uint4(0u, 0u, 0u, 0u);
            continue;
        }
        uint4 x[kConvertColumns / 256];
        float top[kConvertColumns / 256];
#pragma unroll
        for (int j = 0; j < kConvertColumns / 256; ++j)
            if (first + j * 256 < width) {
                x[j] = *reinterpret_cast<const uint4*>(at + j * 256);
                const int64_t u = (first + j * 256 + lane * 8) / kLossUnit;
                top[j] = u < c.units ? c.partial[(u * c.rows + row) * (TWO ? 4 : 2)] : -INFINITY;
            }
        const float4 coef = c.coef[row];
        const int64_t token = LIST ? g.row0[i] + c.row_token[row] : 0;
        const int32_t column = LIST ? 0 : c.row_column[row];
#pragma unroll
        for (int j = 0; j < kConvertColumns / 256; ++j) {
            if (first + j * 256 >= width) break;
            const int col = (int)first + j * 256 + lane * 8;
            const float ref = top[j] == -INFINITY ? 0.f : top[j];
            const float s1 = exp2f(fmaf(ref, k1, -coef.x) - kKeepBits) * coef.y;
            const float b1 = fmaf(ref, k1, -coef.x) - kKeepBits * r1, b2 = fmaf(ref, k2, -coef.z) - kKeepBits * r2;
            uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
                if (TWO) {
                    const float lo = __log2f(f.x), hi = __log2f(f.y);      // 0: -infinity, and 0 again
                    w[e] = bf16x2_rn(coef.y * exp2f(fmaf(lo, r1, b1)) + coef.w * exp2f(fmaf(lo, r2, b2)),
                                     coef.y * exp2f(fmaf(hi, r1, b1)) + coef.w * exp2f(fmaf(hi, r2, b2)));
                } else {
                    w[e] = bf16x2_rn(f.x * s1, f.y * s1);
                }
            }
            // the exact gradient where a target or a teacher has its say
            const auto put = [&](int32_t k, float value) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (k == col + e) {
                        const uint32_t h = f32_to_bf16_rn(value);
                        w[e / 2] = e % 2 ? (w[e / 2] & 0xFFFFu) | h << 16 : (w[e / 2] & 0xFFFF0000u) | h;
                    }
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
            *reinterpret_cast<uint4*>(at + j * 256) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// ---- hidden states' gradients --------------------------------------------------------
template <bool F32>
__global__ void __launch_bounds__(kThreads) k_join(const __grid_constant__ LossGroup g, const __grid_constant__ LossCall c, int splits) {
    pdl_release();
    pdl_acquire();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int first = g.row0[0], last = g.row0[g.n];
    for (int at = first + blockIdx.x * kWarps + warp; at < last; at += gridDim.x * kWarps) {
        const int i = rank_of(g, at), t = at - g.row0[i];
        if (t >= g.tokens[i]) continue;
        const int r = c.token_row[at];
        char* out = static_cast<char*>(g.grad_hidden[i]) + (int64_t)t * c.dim * (F32 ? 4 : 2);
        const bool vec = ((uintptr_t)g.grad_hidden[i] | (uintptr_t)(c.dim * (F32 ? 4 : 2))) % (F32 ? 16 : 8) == 0;
        for (int x = lane * 4; x < c.dim; x += 128) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r >= 0)
                for (int s = 0; s < splits; ++s) {
                    const float4 p = *reinterpret_cast<const float4*>(c.acc + (s * c.rows + g.row0[i] + r) * c.dimp + x);
                    v = make_float4(v.x + p.x, v.y + p.y, v.z + p.z, v.w + p.w);
                }
            const float e[4] = {v.x, v.y, v.z, v.w};
            if (F32) {
                float* o = reinterpret_cast<float*>(out) + x;
                if (vec) *reinterpret_cast<float4*>(o) = v;
                else
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (x + k < c.dim) o[k] = e[k];
            } else {
                uint16_t* o = reinterpret_cast<uint16_t*>(out) + x;
                if (vec) *reinterpret_cast<uint2*>(o) = make_uint2(bf16x2_rn(v.x, v.y), bf16x2_rn(v.z, v.w));
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

cudaError_t launch_loss_scan(const LossGroup& g, const LossCall& c, cudaStream_t stream) {
    return launch_dependent(k_scan, dim3(cap_ctas(g.n)), dim3(kScanThreads), 0, stream, g, c);
}

cudaError_t launch_loss_gather(const LossGroup& g, const LossCall& c, cudaStream_t stream) {
    return launch_dependent(c.dtype == DDP_F32 ? k_gather<true> : k_gather<false>, dim3(warp_grid(g.row0[g.n] - g.row0[0])),
                            dim3(kThreads), 0, stream, g, c);
}

cudaError_t launch_loss_planes(const void* src, void* dst, int64_t rows, const LossCall& c, cudaStream_t stream) {
    return launch_dependent(c.dtype == DDP_F32 ? k_planes<true> : k_planes<false>, dim3(warp_grid(rows)), dim3(kThreads), 0, stream,
                            static_cast<const char*>(src), static_cast<uint16_t*>(dst), rows, c.dim, c.dimp);
}

cudaError_t launch_loss_combine(const LossGroup& g, const LossCall& c, float* loss, cudaStream_t stream) {
    const int64_t blocks = (g.row0[g.n] - g.row0[0]) / kLossBlockRows;
    return launch_dependent(c.two ? k_combine<true> : k_combine<false>, dim3(cap_ctas(std::min<int64_t>(blocks, 2 * sm_count()))),
                            dim3(32 * kCombineWarps), 0, stream, g, c, loss);
}

cudaError_t launch_loss_convert(const LossGroup& g, const LossCall& c, void* piece, int64_t width, cudaStream_t stream) {
    const auto kernel = c.two ? k_convert<true, true> : c.alpha != 0.f ? k_convert<false, true> : k_convert<false, false>;
    const int64_t items = (g.row0[g.n] - g.row0[0]) * ((width + kConvertColumns - 1) / kConvertColumns);
    return launch_dependent(kernel, dim3(warp_grid(items)), dim3(kThreads), 0, stream, g, c, static_cast<uint16_t*>(piece), width);
}

cudaError_t launch_loss_join(const LossGroup& g, const LossCall& c, int splits, cudaStream_t stream) {
    return launch_dependent(c.dtype == DDP_F32 ? k_join<true> : k_join<false>, dim3(warp_grid(g.row0[g.n] - g.row0[0])),
                            dim3(kThreads), 0, stream, g, c, splits);
}

}  // namespace ddpk
