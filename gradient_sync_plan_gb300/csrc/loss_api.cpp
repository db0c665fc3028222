// loss_api.cpp -- the C ABI of the loss head: argument checks, the workspace's
// layout, tensor maps, and the order of a call's launches.
//
// A call of little data is one launch.  Another runs, for all ranks, the teachers'
// lists (distillation) and the gather of learned tokens; then for groups of ranks
// the logits' statistics and their combination into losses; with gradients also,
// for each piece of the vocabulary (or once, where exponentials are kept), its
// logits' gradients and the two products with them, and the join.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <memory>
#include <vector>

#include "ddp_abi_guard.h"
#include "ddp.h"
#include "ddp_spans.h"
#include "ddp_trace.h"
#include "loss_internal.h"

using namespace ddpk;

namespace {

// Bytes of logits' exponentials and gradients that the workspace has room for at most.  Where a rank's tokens by the
// whole vocabulary fit, the exponentials are kept from the loss to the gradients and the logits are computed once, group
// of ranks by group of ranks; else the vocabulary goes in pieces of kPieceBytes.  A piece is written once and read a few
// times, so that it need not fit the L2.
constexpr int64_t kKeepBytes = (int64_t)2 << 30, kPieceBytes = (int64_t)512 << 20;
// Temperatures whose two softmaxes' exponentials come from one another by a power up to this: kept ones' rounding (2^-11) is
// multiplied by it, and 4 leaves it at half of what bf16 rounds off the result (2^-8).
constexpr float kKeepPower = 4.f;
constexpr int64_t kSms = 152;
constexpr int64_t kPieceAlign = 256;              // columns of a piece: a multiple of the tiles'

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// How many parts the depth of the hidden states' gradients is cut into, for at least two tiles an SM and four k
// blocks a part.
int64_t splits_for(int64_t rows, int64_t dim, int64_t width) {
    const int64_t tiles = std::max<int64_t>(1, rows / kTileM * ((dim + kTileN - 1) / kTileN));
    const int64_t blocks = (width + kTileK - 1) / kTileK;
    const int64_t want = std::min((2 * kSms + tiles - 1) / tiles, (blocks + 3) / 4);
    const int64_t part = (blocks + want - 1) / want;
    return (blocks + part - 1) / part;
}

// The widest piece of `bytes` for the rows of a group, balanced over the pieces that the vocabulary then takes.
int64_t piece_width(int64_t bytes, int64_t rows, int64_t vocab, int64_t planes) {
    const int64_t all = round_up(vocab, kPieceAlign);
    int64_t w = std::max(bytes / (2 * planes * std::max<int64_t>(rows, 1)) / kPieceAlign * kPieceAlign, kPieceAlign);
    w = std::min(w, all);
    const int64_t pieces = (all + w - 1) / w;
    return round_up((vocab + pieces - 1) / pieces, kPieceAlign);
}

struct Sizes {
    int64_t counts, factor, done, row_token, token_row, row_column, valid, columns, starts, share, entropy, z, value, partial, coef,
        block_loss, gathered, acc, kept, piece, weights;    // offsets
    int64_t keep_rows;                            // rows of a group whose exponentials are kept
    int64_t acc_bytes, piece_bytes, weights_bytes, total;
};

}  // namespace

struct ddp_loss_head {
    int32_t world = 0, vocab = 0, dim = 0, dtype = 0, max_tokens = 0, max_teacher = 0;
    std::vector<const void*> weights;
    std::vector<void*> grads;
    char* workspace = nullptr;
    Sizes at{};
    std::vector<std::pair<uintptr_t, uintptr_t>> read, written;    // the weights; the workspace and the gradients
    std::vector<CUtensorMap> maps;                                 // of a rank's weights or planes: along and across
    std::vector<CUtensorMap> outs;                                 // of the gradients
    bool stores = false;                                           // whose rows all start on 16-byte boundaries
    int64_t copied = 0;                                            // bytes of a rank's planes in the workspace, 0: none
    int32_t* status = nullptr;
    int device = -1;                                               // that maps and status belong to
};

namespace {

// Whether the products read the weights from the workspace: float32's planes, and bf16 rows that are not whole boxes.
bool is_copied(int32_t dtype, int64_t dim) { return dtype == DDP_F32 || dim % kTileK != 0; }

// Bytes of a logit where exponentials are kept: binary16 that becomes bf16 in place, or a float32 beside three planes.
int64_t kept_bytes(int32_t dtype) { return dtype == DDP_F32 ? 10 : 2; }

int planes_of(int32_t dtype) { return dtype == DDP_F32 ? 3 : 1; }

Sizes layout(int64_t world, int64_t vocab, int64_t dim, int32_t dtype, int64_t max_tokens, int64_t max_teacher, bool grads) {
    Sizes s{};
    const int64_t rows = world * round_up(max_tokens, kLossRowAlign), planes = planes_of(dtype), dimp = round_up(dim, kTileK);
    const int64_t list = max_teacher + 1, units = (vocab + kLossUnit - 1) / kLossUnit;
    const int64_t rank = round_up(max_tokens, kLossRowAlign), group = std::min<int64_t>(world, kLossRanks) * rank;
    int64_t at = 0;
    const auto put = [&](int64_t* offset, int64_t bytes) {
        *offset = at;
        at += round_up(bytes, 256);
    };
    put(&s.counts, 4 * world);
    put(&s.factor, 4 * world);
    put(&s.done, 12);
    put(&s.row_token, 4 * rows);
    put(&s.token_row, 4 * rows);
    put(&s.row_column, 4 * rows);
    put(&s.block_loss, 8 * (rows / kLossBlockRows));
    put(&s.z, 4 * rows * list);
    put(&s.partial, (max_teacher ? 16 : 8) * units * rows);
    if (max_teacher) {
        put(&s.valid, rows);
        put(&s.columns, 4 * rows * list);
        put(&s.starts, 2 * rows * (units + 1));
        put(&s.share, 4 * rows * list);
        put(&s.entropy, 4 * rows);
    }
    put(&s.gathered, 2 * planes * rows * dimp);
    s.weights_bytes = 2 * planes * vocab * dimp;
    put(&s.weights, is_copied(dtype, dim) ? world * s.weights_bytes : 0);
    if (grads) {
        put(&s.value, 4 * rows * list);
        put(&s.coef, 16 * rows);
        // at most 2 kSms / tiles + 1 splits (splits_for), for any number of rows up to these
        s.acc_bytes = 4 * (2 * kSms * kTileM * kTileN + rows * dimp);
        put(&s.acc, s.acc_bytes);
        s.piece_bytes = 2 * planes * group * piece_width(kPieceBytes, group, vocab, planes);
        const int64_t width = round_up(vocab, kPieceAlign), row = kept_bytes(dtype) * width;
        if (rank * row <= kKeepBytes) {
            s.keep_rows = std::min(group, kKeepBytes / row / kLossRowAlign * kLossRowAlign);
            s.piece_bytes = std::max(s.piece_bytes, 2 * planes * s.keep_rows * width);
        }
        put(&s.kept, dtype == DDP_F32 ? 4 * s.keep_rows * width : 0);
        put(&s.piece, s.piece_bytes);
    }
    s.total = at;
    return s;
}

int32_t check_head(int32_t world, int32_t vocab, int32_t dim, int32_t dtype, int32_t max_tokens, int32_t max_teacher) {
    const int32_t st = common_checks(world, 0, dtype);
    if (st) return st;
    if (vocab < 1 || dim < 1 || max_tokens < 1 || max_teacher < 0) return DDP_ERR_INVALID;
    if (vocab > DDP_MAX_VOCAB || dim > DDP_MAX_DIM || max_teacher > DDP_MAX_TEACHER ||
        world * round_up(max_tokens, kLossRowAlign) > ((int64_t)1 << 28) ||
        world * round_up(max_tokens, kLossRowAlign) / kTileM * ((vocab + kTileN - 1) / kTileN) > ((int64_t)1 << 30))   // tiles
        return DDP_ERR_CAPACITY;
    return DDP_OK;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
cudaError_t encoder(EncodeFn* fn) {
    static std::atomic<EncodeFn> found{nullptr};
    *fn = found.load();
    if (*fn) return cudaSuccess;
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || !p) return cudaErrorNotSupported;
    *fn = reinterpret_cast<EncodeFn>(p);
    found.store(*fn);
    return cudaSuccess;
}

// A matrix of bf16 planes [planes][rows][columns], columns a multiple of 64, as [planes][columns / 64][rows][64] in boxes
// of `box_rows` rows and `box_blocks` blocks of columns.
int32_t map_load(CUtensorMap* m, const void* base, int64_t columns, int64_t rows, int64_t planes, int box_rows, int box_blocks) {
    EncodeFn fn;
    const int32_t st = cuda_status(encoder(&fn));
    if (st) return st;
    const cuuint64_t dims[4] = {64, (cuuint64_t)rows, (cuuint64_t)(columns / 64), (cuuint64_t)planes};
    const cuuint64_t strides[3] = {(cuuint64_t)(2 * columns), 128, (cuuint64_t)(2 * columns * rows)};
    const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_blocks, 1}, steps[4] = {1, 1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, steps,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? DDP_OK : cuda_status(cudaErrorInvalidValue);
}
// Boxes of an operand's stage: rows along the depth, or kTileK rows of the depth and their columns across it.
int32_t map_along(CUtensorMap* m, const void* base, int64_t columns, int64_t rows, int64_t planes, int box_rows) {
    return map_load(m, base, columns, rows, planes, box_rows, 1);
}
int32_t map_across(CUtensorMap* m, const void* base, int64_t columns, int64_t rows, int64_t planes, int box_columns) {
    return map_load(m, base, columns, rows, planes, kTileK, box_columns / 64);
}
// [rows][columns] in boxes of 128 rows of 128 bytes, for stores.
int32_t map_out(CUtensorMap* m, const void* base, int32_t dtype, int64_t columns, int64_t rows) {
    EncodeFn fn;
    const int32_t st = cuda_status(encoder(&fn));
    if (st) return st;
    const cuuint64_t dims[2] = {(cuuint64_t)columns, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(columns * elem_bytes(dtype))};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / elem_bytes(dtype)), kTileM}, steps[2] = {1, 1};
    const CUresult r = fn(m, dtype == DDP_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                          const_cast<void*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? DDP_OK : cuda_status(cudaErrorInvalidValue);
}

// What belongs to the device that a head's memory is on, at its first call.
int32_t bind_device(ddp_loss_head* h) {
    int device = 0;
    int32_t st = cuda_status(cudaGetDevice(&device));
    if (st) return st;
    if (h->device >= 0) return device == h->device ? DDP_OK : DDP_ERR_INVALID;
    if ((st = cuda_status(device_status_address(&h->status)))) return st;
    const int64_t dimp = round_up(h->dim, kTileK), planes = planes_of(h->dtype);
    h->maps.resize(2 * h->world);
    h->outs.resize(h->stores ? h->world : 0);
    for (int32_t r = 0; r < h->world; ++r) {
        const void* base = h->copied ? h->workspace + h->at.weights + r * h->copied : static_cast<const void*>(h->weights[r]);
        if ((st = map_along(&h->maps[2 * r], base, dimp, h->vocab, planes, kTileN)) ||
            (st = map_across(&h->maps[2 * r + 1], base, dimp, h->vocab, planes, kTileN)))
            return st;
        if (h->stores && (st = map_out(&h->outs[r], h->grads[r], h->dtype, h->dim, h->vocab))) return st;
    }
    h->device = device;
    return DDP_OK;
}

// The arguments that the four losses share.
struct Args {
    const int32_t* tokens;
    const void* const* hidden;
    int64_t hidden_stride;
    const int64_t* const* targets;
    int64_t ignore_index;
    int32_t reduction;
    float* const* token_losses;
    float* loss;
    // distillation
    int32_t n_teacher = 0;
    const void* const* teacher = nullptr;
    int32_t teacher_dtype = DDP_F32;
    const int64_t* const* indices = nullptr;
    double temperature = 1.0, alpha = 0.0;
    // gradients
    bool grad = false;
    double scale = 1.0;
    int32_t accumulate = 0;
    void* const* grad_hidden = nullptr;
};

int32_t check_args(const ddp_loss_head& h, const Args& a) {
    if (!a.tokens || a.reduction < DDP_LOSS_SUM || a.reduction > DDP_LOSS_WORLD_MEAN) return DDP_ERR_INVALID;
    const bool distill = a.alpha != 0.0;
    if (!a.hidden || (!distill && !a.targets) || a.hidden_stride < h.dim) return DDP_ERR_INVALID;
    if (a.hidden_stride > DDP_MAX_NUMEL / std::max(h.max_tokens, 1)) return DDP_ERR_CAPACITY;
    if (distill) {
        if (!a.teacher || !a.indices || a.n_teacher < 1) return DDP_ERR_INVALID;
        if (a.n_teacher > h.max_teacher) return DDP_ERR_CAPACITY;
        if (a.teacher_dtype != DDP_F32 && a.teacher_dtype != DDP_BF16) return DDP_ERR_INVALID;
        // its square is a factor of the loss, log2 e over it (and a little) of logits
        if (!((float)a.temperature > 0.f) || !std::isfinite((float)(a.temperature * a.temperature)) ||
            !std::isfinite((float)(1.5 / a.temperature)) || !(a.alpha > 0.0 && a.alpha <= 1.0) || !((float)a.alpha > 0.f))
            return DDP_ERR_INVALID;
        if (!a.targets && a.alpha != 1.0) return DDP_ERR_INVALID;
    }
    if (a.grad && (h.grads.empty() || !a.grad_hidden || !std::isfinite((float)a.scale))) return DDP_ERR_INVALID;
    int32_t st = check_ptr(a.loss, 4);
    if (st) return st;
    const int64_t es = elem_bytes(h.dtype), ts = elem_bytes(a.teacher_dtype);
    std::vector<Span> written(h.written), read(h.read);
    written.push_back(span_of(a.loss, 4 * (int64_t)h.world));
    for (int32_t r = 0; r < h.world; ++r) {
        const int64_t n = a.tokens[r];
        if (n < 0) return DDP_ERR_INVALID;
        if (n > h.max_tokens) return DDP_ERR_CAPACITY;
        if (n == 0) continue;
        if ((st = check_ptr(a.hidden[r], es))) return st;
        read.push_back(span_of(a.hidden[r], ((n - 1) * a.hidden_stride + h.dim) * es));
        if (a.targets) {
            if ((st = check_ptr(a.targets[r], 8))) return st;
            read.push_back(span_of(a.targets[r], 8 * n));
        }
        if (distill) {
            if ((st = check_ptr(a.teacher[r], ts)) || (st = check_ptr(a.indices[r], 8))) return st;
            read.push_back(span_of(a.teacher[r], ts * n * a.n_teacher));
            read.push_back(span_of(a.indices[r], 8 * n * a.n_teacher));
        }
        if (a.token_losses && a.token_losses[r]) {
            if ((st = check_ptr(a.token_losses[r], 4))) return st;
            written.push_back(span_of(a.token_losses[r], 4 * n));
        }
        if (a.grad) {
            if ((st = check_ptr(a.grad_hidden[r], es))) return st;
            written.push_back(span_of(a.grad_hidden[r], n * h.dim * es));
        }
    }
    if (any_overlap(&written)) return DDP_ERR_INVALID;
    for (const Span& s : read)
        if (hits_any(written, s)) return DDP_ERR_INVALID;
    return DDP_OK;
}

int32_t run(ddp_loss_head* h, const Args& a, cudaStream_t stream) {
    int32_t st = check_args(*h, a);
    if (st) return st;
    if ((st = bind_device(h))) return st;
    const bool distill = a.alpha != 0.0;
    LossCall c{};
    c.vocab = h->vocab;
    c.dim = h->dim;
    c.dimp = (int32_t)round_up(h->dim, kTileK);
    c.dtype = h->dtype;
    c.planes = planes_of(h->dtype);
    c.teacher_dtype = a.teacher_dtype;
    c.n_teacher = a.n_teacher;
    c.list = distill ? a.n_teacher + (a.targets ? 1 : 0) : 1;
    c.units = (h->vocab + kLossUnit - 1) / kLossUnit;
    c.reduction = a.reduction;
    c.alpha = (float)a.alpha;
    c.temperature = (float)a.temperature;
    c.inv_temperature = (float)(1.0 / a.temperature);
    c.two = distill && c.alpha < 1.f && c.temperature != 1.f;
    // 1 + cut itself may lie between two floats: it multiplies in double here, and by fmaf in the kernels
    const double cut = (double)kCutPerStep * (c.dimp / 16), bits = 1.4426950408889634 * (1.0 + cut);
    c.cut = (float)cut;
    c.k2 = (float)(bits / a.temperature);
    c.k1 = c.two ? (float)bits : c.k2;
    c.hidden_stride = a.hidden_stride;
    c.ignore_index = a.ignore_index;
    c.scale = (float)a.scale;
    char* w = h->workspace;
    const Sizes& at = h->at;
    c.counts = reinterpret_cast<int32_t*>(w + at.counts);
    c.factor = reinterpret_cast<float*>(w + at.factor);
    c.done = reinterpret_cast<int32_t*>(w + at.done);
    c.next = c.done + 1;
    c.row_token = reinterpret_cast<int32_t*>(w + at.row_token);
    c.token_row = reinterpret_cast<int32_t*>(w + at.token_row);
    c.row_column = reinterpret_cast<int32_t*>(w + at.row_column);
    c.valid = reinterpret_cast<uint8_t*>(w + at.valid);
    c.columns = reinterpret_cast<int32_t*>(w + at.columns);
    c.starts = reinterpret_cast<uint16_t*>(w + at.starts);
    c.share = reinterpret_cast<float*>(w + at.share);
    c.entropy = reinterpret_cast<float*>(w + at.entropy);
    c.z = reinterpret_cast<float*>(w + at.z);
    c.value = a.grad ? reinterpret_cast<float*>(w + at.value) : nullptr;
    c.partial = reinterpret_cast<float*>(w + at.partial);
    c.coef = reinterpret_cast<float4*>(w + at.coef);
    c.block_loss = reinterpret_cast<double*>(w + at.block_loss);
    c.gathered = w + at.gathered;
    c.acc = reinterpret_cast<float*>(w + at.acc);
    c.status = h->status;

    // the groups of ranks, and where their rows are
    const int64_t vocab_width = round_up(h->vocab, kPieceAlign);
    const bool may_keep = a.grad && (!c.two || std::max(c.temperature, c.inv_temperature) <= kKeepPower);
    const int64_t keep_rows = may_keep ? at.keep_rows : 0;
    std::vector<LossGroup> groups;
    int64_t rows = 0;
    for (int32_t r = 0; r < h->world; ++r) {
        const int32_t n = a.tokens[r];
        const int64_t mine = round_up(n, kLossRowAlign);
        if (groups.empty() || groups.back().n == kLossRanks ||
            (keep_rows > 0 && rows > groups.back().row0[0] && rows + mine - groups.back().row0[0] > keep_rows)) {
            groups.push_back(LossGroup{});
            groups.back().world = h->world;
            groups.back().first = r;
            groups.back().row0[0] = (int32_t)rows;
        }
        LossGroup& g = groups.back();
        const int i = g.n++;
        g.tokens[i] = n;
        g.hidden[i] = a.hidden[r];
        g.targets[i] = a.targets ? a.targets[r] : nullptr;
        g.teacher[i] = distill ? a.teacher[r] : nullptr;
        g.indices[i] = distill ? a.indices[r] : nullptr;
        g.token_losses[i] = a.token_losses ? a.token_losses[r] : nullptr;
        g.grad_hidden[i] = a.grad ? a.grad_hidden[r] : nullptr;
        rows += mine;
        g.row0[i + 1] = (int32_t)rows;
    }
    c.rows = std::max<int64_t>(rows, kLossRowAlign);

    if (groups.size() == 1 && loss_is_small(groups[0], c)) {
        LossSmall m{};
        for (int32_t r = 0; r < h->world; ++r) {
            m.weights[r] = h->weights[r];
            m.grads[r] = a.grad ? h->grads[r] : nullptr;
        }
        m.grad = a.grad;
        m.accumulate = a.accumulate;
        return cuda_status(launch_loss_small(groups[0], c, m, a.loss, stream));
    }
    for (const LossGroup& g : groups)
        if ((distill && (st = cuda_status(launch_loss_teacher(g, c, stream)))) || (st = cuda_status(launch_loss_gather(g, c, stream))))
            return st;
    if (h->copied)
        for (const LossGroup& g : groups) {
            LossWeights p{};
            p.n = g.n;
            std::copy(h->weights.begin() + g.first, h->weights.begin() + g.first + g.n, p.weights);
            if ((st = cuda_status(launch_loss_planes(p, w + at.weights + g.first * h->copied, h->copied, c, stream)))) return st;
        }

    LossGemm m{};
    m.c = c;
    m.limit_ns = std::max(wait_limit_ns(), 2000000000ull);
    m.accumulate = a.accumulate;
    CUtensorMap hidden[2];                 // along, across
    if ((st = map_along(&hidden[0], c.gathered, c.dimp, c.rows, c.planes, kTileM)) ||
        (st = map_across(&hidden[1], c.gathered, c.dimp, c.rows, c.planes, kTileN)))
        return st;
    if (a.grad) m.store = h->stores && !a.accumulate;
    for (const LossGroup& g : groups) {
        const int64_t span = g.row0[g.n] - g.row0[0];
        m.n = g.n;
        m.first = g.first;
        std::copy(g.row0, g.row0 + kLossRanks + 1, m.row0);
        for (int i = 0; i < g.n; ++i) {
            m.grads[i] = a.grad ? h->grads[g.first + i] : nullptr;
            if (a.grad && h->stores) m.out[i] = h->outs[g.first + i];
        }
        const bool keep = span > 0 && span <= keep_rows;
        const int64_t width = !a.grad || keep ? vocab_width : piece_width(at.piece_bytes, span, h->vocab, c.planes);
        if (a.grad) {
            m.splits = (int32_t)splits_for(c.rows, c.dim, std::min<int64_t>(width, h->vocab));
            const int64_t blocks = (std::min<int64_t>(width, h->vocab) + kTileK - 1) / kTileK;
            m.split_blocks = (int32_t)((blocks + m.splits - 1) / m.splits);
            if ((st = map_out(&m.acc, c.acc, DDP_F32, c.dimp, m.splits * c.rows))) return st;
            if (span > 0 && ((st = map_along(&m.piece, w + at.piece, width, span, c.planes, kTileM)) ||
                             (st = map_across(&m.piece_across, w + at.piece, width, span, c.planes, kTileM)) ||
                             (st = map_out(&m.piece_out, w + at.piece, DDP_BF16, width, span * c.planes)) ||
                             (st = map_out(&m.keep_out, h->dtype == DDP_F32 ? w + at.kept : w + at.piece, h->dtype, width, span))))
                return st;
        }
        const auto operands = [&](bool across) {
            m.hidden = hidden[across];
            for (int i = 0; i < g.n; ++i) m.weights[i] = h->maps[2 * (g.first + i) + across];
        };
        const auto products = [&](LossPhase phase) {
            m.stall = take_planted_stall();
            return cuda_status(launch_loss_gemm(phase, m, stream));
        };
        operands(false);
        if (span > 0) {
            m.piece0 = 0;
            m.width = h->vocab;
            if ((st = products(keep ? LossPhase::kKeep : LossPhase::kStats))) return st;
        }
        if ((st = cuda_status(launch_loss_combine(g, c, a.loss, stream)))) return st;
        if (!a.grad) continue;
        for (int64_t v = 0; v < h->vocab; v += width) {
            m.piece0 = (int32_t)v;
            m.width = (int32_t)std::min<int64_t>(width, h->vocab - v);
            m.add = v > 0;
            operands(false);
            if (keep) st = cuda_status(launch_loss_convert(g, c, h->dtype == DDP_F32 ? w + at.kept : w + at.piece, w + at.piece, width, stream));
            else st = products(LossPhase::kGrad);
            operands(true);
            if (st || (st = products(LossPhase::kProducts))) return st;
        }
        if (span > 0 && (st = cuda_status(launch_loss_join(g, c, m.splits, stream)))) return st;
    }
    return DDP_OK;
}

}  // namespace

extern "C" {

int32_t ddp_loss_head_workspace_bytes(int32_t world, int32_t vocab, int32_t dim, int32_t dtype, int32_t max_tokens,
                                      int32_t max_teacher, int32_t with_grads, int64_t* bytes) try {
    DDP_TRACE_CALL();
    const int32_t st = check_head(world, vocab, dim, dtype, max_tokens, max_teacher);
    if (st) return st;
    if (!bytes) return DDP_ERR_INVALID;
    *bytes = layout(world, vocab, dim, dtype, max_tokens, max_teacher, with_grads != 0).total;
    return DDP_OK;
} DDP_ABI_CATCH

int32_t ddp_loss_head_create(int32_t world, const void* const* weights, void* const* grads, int32_t vocab, int32_t dim,
                             int32_t dtype, int32_t max_tokens, int32_t max_teacher, void* workspace,
                             int64_t workspace_bytes, ddp_loss_head** out) try {
    DDP_TRACE_CALL();
    if (!out) return DDP_ERR_INVALID;
    *out = nullptr;
    int32_t st = check_head(world, vocab, dim, dtype, max_tokens, max_teacher);
    if (st) return st;
    if (!weights) return DDP_ERR_INVALID;
    if ((st = check_ptr(workspace, 256))) return st;
    std::unique_ptr<ddp_loss_head> h(new ddp_loss_head());
    h->world = world;
    h->vocab = vocab;
    h->dim = dim;
    h->dtype = dtype;
    h->max_tokens = max_tokens;
    h->max_teacher = max_teacher;
    h->workspace = static_cast<char*>(workspace);
    h->at = layout(world, vocab, dim, dtype, max_tokens, max_teacher, grads != nullptr);
    if (workspace_bytes < h->at.total) return DDP_ERR_CAPACITY;
    const int64_t es = elem_bytes(dtype), bytes = (int64_t)vocab * dim * es;
    h->written.push_back(span_of(workspace, h->at.total));
    for (int32_t r = 0; r < world; ++r) {
        if ((st = check_ptr(weights[r], is_copied(dtype, dim) ? es : 16))) return st;
        h->weights.push_back(weights[r]);
        h->read.push_back(span_of(weights[r], bytes));
        if (!grads) continue;
        if ((st = check_ptr(grads[r], es))) return st;
        h->grads.push_back(grads[r]);
        h->written.push_back(span_of(grads[r], bytes));
    }
    if (is_copied(dtype, dim)) h->copied = h->at.weights_bytes;
    h->stores = grads != nullptr && dim * es % 16 == 0;
    for (void* p : h->grads) h->stores &= reinterpret_cast<uintptr_t>(p) % 16 == 0;
    if (any_overlap(&h->written)) return DDP_ERR_INVALID;
    for (const Span& s : h->read)
        if (hits_any(h->written, s)) return DDP_ERR_INVALID;
    *out = h.release();
    return DDP_OK;
} DDP_ABI_CATCH

int32_t ddp_cross_entropy(ddp_loss_head* head, const int32_t* tokens, const void* const* hidden, int64_t hidden_stride,
                          const int64_t* const* targets, int64_t ignore_index, int32_t reduction,
                          float* const* token_losses, float* loss, void* stream) try {
    DDP_TRACE_CALL();
    if (!head) return DDP_ERR_INVALID;
    return run(head, Args{tokens, hidden, hidden_stride, targets, ignore_index, reduction, token_losses, loss},
               (cudaStream_t)stream);
} DDP_ABI_CATCH

int32_t ddp_cross_entropy_grad(ddp_loss_head* head, const int32_t* tokens, const void* const* hidden,
                               int64_t hidden_stride, const int64_t* const* targets, int64_t ignore_index,
                               int32_t reduction, double scale, int32_t accumulate, float* const* token_losses,
                               float* loss, void* const* grad_hidden, void* stream) try {
    DDP_TRACE_CALL();
    if (!head) return DDP_ERR_INVALID;
    Args a{tokens, hidden, hidden_stride, targets, ignore_index, reduction, token_losses, loss};
    a.grad = true;
    a.scale = scale;
    a.accumulate = accumulate;
    a.grad_hidden = grad_hidden;
    return run(head, a, (cudaStream_t)stream);
} DDP_ABI_CATCH

int32_t ddp_distill(ddp_loss_head* head, const int32_t* tokens, const void* const* hidden, int64_t hidden_stride,
                    int32_t n_teacher, const void* const* teacher, int32_t teacher_dtype, const int64_t* const* indices,
                    double temperature, double alpha, const int64_t* const* targets, int64_t ignore_index,
                    int32_t reduction, float* const* token_losses, float* loss, void* stream) try {
    DDP_TRACE_CALL();
    if (!head || !((float)alpha > 0.f)) return DDP_ERR_INVALID;
    return run(head,
               Args{tokens, hidden, hidden_stride, targets, ignore_index, reduction, token_losses, loss, n_teacher, teacher,
                    teacher_dtype, indices, temperature, alpha},
               (cudaStream_t)stream);
} DDP_ABI_CATCH

int32_t ddp_distill_grad(ddp_loss_head* head, const int32_t* tokens, const void* const* hidden, int64_t hidden_stride,
                         int32_t n_teacher, const void* const* teacher, int32_t teacher_dtype,
                         const int64_t* const* indices, double temperature, double alpha,
                         const int64_t* const* targets, int64_t ignore_index, int32_t reduction, double scale,
                         int32_t accumulate, float* const* token_losses, float* loss, void* const* grad_hidden,
                         void* stream) try {
    DDP_TRACE_CALL();
    if (!head || !((float)alpha > 0.f)) return DDP_ERR_INVALID;
    return run(head,
               Args{tokens, hidden, hidden_stride, targets, ignore_index, reduction, token_losses, loss, n_teacher, teacher,
                    teacher_dtype, indices, temperature, alpha, true, scale, accumulate, grad_hidden},
               (cudaStream_t)stream);
} DDP_ABI_CATCH

int32_t ddp_loss_head_destroy(ddp_loss_head* head) try {
    DDP_TRACE_CALL();
    delete head;
    return DDP_OK;
} DDP_ABI_CATCH

}  // extern "C"
