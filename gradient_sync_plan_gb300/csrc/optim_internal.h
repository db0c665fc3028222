// optim_internal.h -- what the gradient norm, clipping and AdamW sources share
// on the host side.  Not part of the C ABI (see include/ddp.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <memory>
#include <vector>

#include "ddp_internal.h"

namespace ddpk {

// ---- tables in device memory (grad_norm.cu) ----------------------------------
// A kernel's table travels in its parameters while one launch takes it.  Where
// it would take several launches for little data, a handle keeps it in its
// workspace instead, written there by launches of its own before the first use.
struct DeviceTable {
    std::vector<char> image;                   // tile ends, then entries
    int64_t entries_at = 0;                    // byte offset of the entries
    int64_t more_at = 0;                       // and of what follows them
};
// Whether entries that take `launches` launches, moving `bytes`, do better as one
// from a table in device memory: another launch costs some 5 us, the table's
// loads some 5 % of a large launch.
inline bool table_on_device(int64_t launches, int64_t bytes) {
    return launches > 1 && bytes < (launches - 1) * ((int64_t)512 << 20);
}
// Workspace for the table of `entries` entries of `entry` bytes, and its start
// behind the `used` bytes before it.
inline int64_t table_offset(int64_t used) { return (used + 255) / 256 * 256; }
inline int64_t table_space(int64_t used, int64_t entries, int64_t entry) {
    return table_offset(used) + (4 * entries + 15) / 16 * 16 + (entries * entry + 15) / 16 * 16;
}
cudaError_t upload_table(const DeviceTable& t, void* device, cudaStream_t stream);

// ---- norm and clip (grad_norm.cu) ---------------------------------------
// A run of contiguous gradient bytes of one rank: what the norm and clip
// kernels walk.  Tensors that lie back to back in memory are one range.
struct GradRange {
    char* ptr;
    int64_t bytes;
    int32_t rank;
};

// Bytes of a tile of the norm and clip kernels.  Tiles start at 128-byte
// boundaries of memory, so a range has at most one more than bytes / kNormTile
// rounded up.  A norm block takes a run of them: as many as make kNormBlocks
// blocks (eight on each of 152 SMs) while kNormOneWave are enough for that, else
// kNormRun.
constexpr int64_t kNormTile = 16384;
constexpr int64_t kNormAlign = 128;
constexpr int64_t kNormRun = 4;
constexpr int64_t kNormOneWave = 16;
constexpr int64_t kNormBlocks = 8 * 152;

// The kernels' tables, filled once for ranges sorted by rank.
struct RangePlan;
std::shared_ptr<const RangePlan> make_range_plan(const GradRange* ranges, int64_t n, int ranks);
constexpr int64_t kRangeEntry = 24;

// How a launch of partials ends: where there are few, its last block adds them
// itself (counter: a word that is zero between launches); NULL: it does not.
constexpr int kFinishRanks = 16;
constexpr int32_t kFinishPartials = 1280;
struct NormFinish {
    uint32_t* counter;
    float* norms;
    int32_t ranks, copies;                     // norms[r * copies ..] receive rank r's
    int32_t first[kFinishRanks + 1];           // rank r's partials are first[r] .. first[r + 1]
};

// Where a norm's launches put things: the workspace's counter, which the first
// launch finds zero, and its partials.
struct NormSpace {
    uint32_t* counter;
    double* partials;
    char* table;                               // for a DeviceTable
};
constexpr int64_t kNormSpaceHead = 16;         // bytes before the partials

// norms[r * copies ..] = sqrt(sum of squares of rank r's ranges).
cudaError_t launch_norm(const RangePlan& plan, int dtype, NormSpace ws, int copies, float* norms, cudaStream_t stream);
cudaError_t launch_clip(const RangePlan& plan, int dtype, NormSpace ws, const float* norms, float max_norm,
                        cudaStream_t stream);
// The plan's table, if it belongs in device memory (else null): to be uploaded
// to ws.table before the first launch.
const DeviceTable* range_plan_table(const RangePlan& plan);
NormFinish norm_finish(NormSpace ws, const int32_t* rank_first, int ranks, int copies, float* norms, bool one_launch);
// Partials that a launch left, into norms.
cudaError_t launch_norm_final(const double* partials, const int32_t* rank_first, int ranks, int copies, float* norms,
                              cudaStream_t stream);

// ---- view sync with the norm in its epilogue (sync_norm.cu) ----------------
// One bucket member: its elements, its place in its bucket, its bucket's chunk
// length and its `world` pointers.
struct SyncMember {
    int64_t numel, offset, clen;
    void* const* ptrs;
};
// Vectors a thread takes of a tile when a rank's members have numel elements.
int sync_norm_vecs(int world, int64_t numel, int dtype);
// The kernel's tables, filled once.  dtype: a ddp_dtype or one of the hooks'
// (kDtypeHook, kDtypeHook16).
struct SyncPlan;
std::shared_ptr<const SyncPlan> make_sync_plan(int world, const SyncMember* members, int64_t n, int vecs, int dtype,
                                               DivSpec div);
const DeviceTable* sync_plan_table(const SyncPlan& plan);
constexpr int64_t kSyncEntry = 32;             // and 8 a rank
cudaError_t launch_sync_norm(const SyncPlan& plan, NormSpace ws, float* norms, cudaStream_t stream);

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
int64_t adamw_tiles(const AdamWItem& it);
// The kernel's tables, filled once.
struct AdamWPlan;
std::shared_ptr<const AdamWPlan> make_adamw_plan(const AdamWItem* items, int64_t n, int grad_dtype, bool copies);
const DeviceTable* adamw_plan_table(const AdamWPlan& plan);
constexpr int64_t kAdamWEntry = 56;
// norms may be null (no clipping).  steps[world] is read, and advanced for the
// ranks that were updated; arrivals is one word, zero between calls; table is
// where the plan's device table is, if it has one.
cudaError_t launch_adamw(const AdamWPlan& plan, const char* table, int world, int grad_dtype, bool copies,
                         const AdamWScalars& s, const float* norms, int32_t* steps, int32_t* arrivals, cudaStream_t stream);

}  // namespace ddpk
