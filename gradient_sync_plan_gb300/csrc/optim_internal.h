// optim_internal.h -- what the gradient norm, clipping and AdamW sources share
// on the host side.  Not part of the C ABI (see include/ddp.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <vector>

#include "ddp_internal.h"

namespace ddpk {

// ---- norm and clip (grad_norm.cu) ---------------------------------------
// A run of contiguous gradient bytes of one rank: what the norm and clip
// kernels walk.  Tensors that lie back to back in memory are one range.
struct GradRange {
    char* ptr;
    int64_t bytes;
    int32_t rank;
};

// Bytes that one block of the norm and clip kernels takes.  Tiles start at
// 128-byte boundaries of memory, so a range has at most one more than
// bytes / kNormTile rounded up.
constexpr int64_t kNormTile = 16384;
constexpr int64_t kNormAlign = 128;
int64_t range_tiles(const void* ptr, int64_t bytes);

// Partial sums of squares (one double a tile, in the order of the ranges,
// which are sorted by rank), then norms[r] = sqrt(sum of rank r's partials).
// rank_first[r] .. rank_first[r + 1] are rank r's partials.
cudaError_t launch_norm_partials(const GradRange* ranges, int64_t n, int dtype, double* partials, cudaStream_t stream);
// Each of `ranks` norms is written `copies` times, norms[r * copies ..].
cudaError_t launch_norm_final(const double* partials, const int32_t* rank_first, int ranks, int copies, float* norms,
                              cudaStream_t stream);
cudaError_t launch_clip(const GradRange* ranges, int64_t n, int dtype, const float* norms, float max_norm,
                        cudaStream_t stream);

// ---- view sync with the norm in its epilogue (sync_norm.cu) ----------------
// One bucket member: its elements, its place in its bucket, its bucket's chunk
// length and its `world` pointers.
struct SyncMember {
    int64_t numel, offset, clen;
    void* const* ptrs;
};
// Vectors a thread takes of a tile when a rank's members have numel elements,
// and the tiles (one partial each) of one member.
int sync_norm_vecs(int world, int64_t numel, int dtype);
int64_t sync_norm_tiles(int world, const SyncMember& m, int vecs, int dtype);
// dtype: a ddp_dtype or one of the hooks' (kDtypeHook, kDtypeHook16).
cudaError_t launch_sync_norm(int world, const SyncMember* members, int64_t n, int vecs, int dtype, DivSpec div,
                             double* partials, cudaStream_t stream);

// ---- AdamW (adamw.cu) ------------------------------------------------------
// One tensor of one rank.  g is float32 or bf16 (the call's grad dtype), copy
// bf16 or null, the others float32.
struct AdamWItem {
    float* p;
    float* m;
    float* v;
    const void* g;
    void* copy;
    int64_t numel;
    int32_t rank;
    int32_t decay;         // 0: this tensor has no weight decay
};
struct AdamWScalars {
    float lr, beta1, one_minus_beta1, ln_beta1, beta2, one_minus_beta2, ln_beta2, eps, lr_decay, max_norm;
};
int64_t adamw_tiles(const AdamWItem& it, int grad_dtype);
// norms may be null (no clipping).  steps[world] is read, and advanced for the
// ranks that were updated; arrivals is one word, zero between calls.
cudaError_t launch_adamw(const AdamWItem* items, int64_t n, int world, int grad_dtype, bool copies, AdamWScalars s,
                         const float* norms, int32_t* steps, int32_t* arrivals, cudaStream_t stream);

}  // namespace ddpk
