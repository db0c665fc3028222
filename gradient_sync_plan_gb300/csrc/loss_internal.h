// loss_internal.h -- what the loss head's sources share on the host side and in
// their kernels' parameters.  Not part of the C ABI (see include/ddp.h).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ddp_internal.h"

namespace ddpk {

// Ranks of one launch; more take further launches.
constexpr int kLossRanks = 16;
// A rank's learned tokens are gathered into rows of its own, from a multiple of kLossRowAlign on.
constexpr int kLossRowAlign = 256;
// Columns of a partial softmax statistic and of a bin of listed columns.
constexpr int kLossUnit = 128;
// Tile of the products: rows, columns, depth of a shared-memory stage.
constexpr int kTileM = 128, kTileN = 256, kTileK = 64;

// The tensor cores cut a sum's low bits where they add 16 products to it, so sums come out a little small: by 1.6e-8 of
// the result a step of 16 where the sum grows evenly or wanders (measured on sums of 256 to 16384 products of either
// sign, 1.4e-8 to 1.6e-8; of one sign 2.5e-8 and more).  Logits and float32 gradients, each part of a depth taken out of
// tensor memory by itself, are scaled back by that: 4096 products' mean error of 4.0e-6 becomes 0.1e-6, of products of one
// sign 1.4e-5 becomes 1.0e-5.
constexpr float kCutPerStep = 1.6e-8f;

// One group of ranks as the row kernels see it.  Rows are numbered through all
// ranks: rank i of the group has rows row0[i] .. row0[i + 1], its first counts[i]
// hold its learned tokens.
struct LossGroup {
    int32_t n;                            // ranks
    int32_t world, first;                 // of all, and the group's first
    int32_t row0[kLossRanks + 1];
    int32_t tokens[kLossRanks];
    const void* hidden[kLossRanks];
    const int64_t* targets[kLossRanks];   // null: none
    const void* teacher[kLossRanks];
    const int64_t* indices[kLossRanks];
    float* token_losses[kLossRanks];      // null: not wanted
    void* grad_hidden[kLossRanks];
};

// The call's constants, and the workspace's arrays (by row or token of all ranks).
struct LossCall {
    int32_t vocab, dim, dimp;             // dimp: dim rounded up to kTileK, a gathered row's length
    int32_t dtype, planes;                // bf16 planes of an operand: 1, or 3 for float32
    int32_t teacher_dtype, n_teacher, list;   // list: columns a token lists (1: its target)
    int32_t units;                        // statistics units of the vocabulary
    int32_t reduction, two;               // two: softmaxes of two temperatures
    int64_t hidden_stride, ignore_index;
    float inv_temperature, temperature;   // of the distillation
    float alpha;                          // its share; 0: cross entropy alone
    float cut;                            // of the tensor cores' logits' sums (kCutPerStep)
    float k1, k2;                         // from a difference of them to bits: log2 e (1 + cut), of the softmax or the first
                                          // of two, and at the temperature
    float scale;                          // of the gradients
    int64_t rows;                         // rows of all ranks

    int32_t* counts;                      // [world]
    int32_t* done;                        // blocks of a combine launch that are through
    int32_t* next;                        // [2] tiles taken of a products' launch, and blocks that are through
    int32_t* row_token;                   // [rows] the token (of its rank) that a row holds
    int32_t* token_row;                   // [rows] the row (of its rank) of a token, -1: not learned
    int32_t* row_column;                  // [rows] target's column
    uint8_t* valid;                       // [rows] by token: learned (distillation)
    int32_t* columns;                     // [rows][list] by token, ascending
    uint16_t* starts;                     // [rows][units + 1] by token: entries before a unit
    float* share;                         // [rows][list] by token: teacher's probability of the entry
    float* entropy;                       // [rows] by token: sum of q log q
    float* z;                             // [rows][list] the tensor cores' logits at the listed columns
    float* value;                         // [rows][list] gradients there, without the factor
    float* partial;                       // [units][rows] float2, or float4 for two temperatures: the tensor cores' largest
                                          // logit, and the sum of exponentials relative to it but for one of the largest
    float* factor;                        // [world] of the gradients: scale and reduction
    float4* coef;                         // [rows] {largest logit, share over the sum of exponentials relative to it, -, the
                                          // same at the temperature}
    double* block_loss;                   // [rows / kLossBlockRows]
    void* gathered;                       // [planes][rows][dimp] bf16
    float* acc;                           // [splits][rows][dimp]
    int32_t* status;                      // the device status word
};
constexpr int kLossBlockRows = 32;        // rows of a combine block

// Products.  kStats: logits' statistics and listed logits.  kKeep: those, and the logits' exponentials relative to
// their unit's largest: of bf16 operands binary16 scaled by 2^kKeepBits, of float32 ones as they are.  kGrad: logits' gradients of a
// piece of the vocabulary, to `piece`.  kProducts: the piece's share of the hidden states' gradients
// (added to acc) and its rows of the weights' gradients.
enum class LossPhase { kStats = 0, kGrad = 1, kProducts = 2, kKeep = 3 };
constexpr int kKeepBits = 15;             // largest of a unit: 2^15, below binary16's 65504

struct LossGemm {
    // loads, in boxes of what a block's stage takes along the depth (rows of an operand) or, where the phase's product
    // is over their rows, across it
    CUtensorMap hidden;                   // gathered rows; across for kProducts
    CUtensorMap piece, piece_across;      // [planes][rows of the group][piece columns] bf16
    CUtensorMap weights[kLossRanks];      // across for kProducts
    // stores, in boxes of 128 rows of 128 bytes
    CUtensorMap piece_out, keep_out, acc; // acc: [splits * rows][dimp] float32
    CUtensorMap out[kLossRanks];          // the weights' gradients, where `store`
    void* grads[kLossRanks];
    int32_t row0[kLossRanks + 1];
    int32_t n, first;
    int32_t piece0, width;                // the piece's first column and its columns
    int32_t splits, split_blocks;         // of the hidden states' gradients: parts of the piece's depth, their k blocks
    int32_t add;                          // add to acc (else write)
    int32_t accumulate;                   // add to the weights' gradients
    int32_t store;                        // the copy engine writes them: 16-byte aligned rows, not accumulated
    unsigned long long limit_ns;
    int64_t stall;                        // the tile from which on its block loads nothing (ddp_plant_stall), -1: none
    LossCall c;
};
static_assert(sizeof(LossGemm) < 8192, "travels in the kernel's parameters");

cudaError_t launch_loss_gemm(LossPhase phase, const LossGemm& g, cudaStream_t stream);

// ---- rows (loss_rows.cu) ---------------------------------------------------
// Teachers' entries: sorted lists, probabilities, which tokens are learned.
cudaError_t launch_loss_teacher(const LossGroup& g, const LossCall& c, cudaStream_t stream);
// Which tokens are learned, and their hidden states into rows; the rows that pad a rank's last are zeroed.
cudaError_t launch_loss_gather(const LossGroup& g, const LossCall& c, cudaStream_t stream);
// The weights of a group's ranks as [planes][vocab][dimp] bf16, zeros behind dim, `bytes` a rank.
struct LossWeights {
    int32_t n;
    const void* weights[kLossRanks];
};
cudaError_t launch_loss_planes(const LossWeights& m, void* dst, int64_t bytes, const LossCall& c, cudaStream_t stream);
// Partial statistics to losses and to the gradients' coefficients.
cudaError_t launch_loss_combine(const LossGroup& g, const LossCall& c, float* loss, cudaStream_t stream);
// Kept exponentials [rows of the group][width] to the logits' gradients' planes in `piece`; bf16: in place, `kept` is `piece`.
cudaError_t launch_loss_convert(const LossGroup& g, const LossCall& c, const void* kept, void* piece, int64_t width,
                                cudaStream_t stream);
// acc's splits to the hidden states' gradients, zeros for tokens that are not learned.
cudaError_t launch_loss_join(const LossGroup& g, const LossCall& c, int splits, cudaStream_t stream);

// ---- little data (loss_small.cu) --------------------------------------------
struct LossSmall {
    const void* weights[kLossRanks];
    void* grads[kLossRanks];
    int32_t grad, accumulate;
    int32_t most_tokens;                  // of a rank
};
// Elements of the weights (their floats fit shared memory beside the rest), multiplications of a rank's product, and
// teachers' entries of all ranks up to which one launch does everything.  Against the launches of the general way, in us:
// 2^18 multiplications (16 tokens, 256 x 64) 11.5 and 16.9 for a loss, 25.0 and 28.4 with gradients; 2^19 (64 tokens,
// 256 x 32) 20.7 and 18.9, 46.2 and 31.0.
constexpr int64_t kSmallWeights = 16384, kSmallWork = 1 << 18, kSmallEntries = 16384;
bool loss_is_small(const LossGroup& g, const LossCall& c);
cudaError_t launch_loss_small(const LossGroup& g, const LossCall& c, LossSmall m, float* loss, cudaStream_t stream);

// Lets a kernel take this much dynamic shared memory, once a process and device.
cudaError_t allow_shared_memory(const void* kernel, int bytes);

#ifdef __CUDACC__
// The device status word: DDP_ERR_INVALID leaves a DDP_ERR_TIMEOUT as it is, whose buffers hold partial results.
__device__ __forceinline__ void report_invalid(int32_t* status) { atomicCAS(status, (int32_t)DDP_OK, (int32_t)DDP_ERR_INVALID); }
#endif

// The address of the device status word, the TMA kernels' wait limit, and a tile that a test has planted for the next
// launch's loads to stop at, or -1 (ring_tma.cu).
cudaError_t device_status_address(int32_t** word);
unsigned long long wait_limit_ns();
long long take_planted_stall();

}  // namespace ddpk
