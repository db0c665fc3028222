// optim_api.cpp -- the C ABI of the gradient norm, clipping, the sync that
// returns the norm, and AdamW: argument checks, tables, launches.
//
// A grad set or an AdamW handle checks its tensors once, when it is made, and
// keeps the table that its launches pass to the kernels; a call then costs its
// launches and nothing that grows with the number of tensors but the table's
// copy into them.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <memory>
#include <utility>
#include <vector>

#include "ddp_abi_guard.h"
#include "ddp.h"
#include "ddp_trace.h"
#include "optim_internal.h"

using namespace ddpk;

struct ddp_grad_set {
    int32_t world = 0, dtype = 0;
    std::shared_ptr<const RangePlan> plan;
    std::vector<std::pair<uintptr_t, uintptr_t>> spans;        // the memory of the tensors and the workspace, sorted
    NormSpace space{nullptr, nullptr, nullptr};
    bool ready = false;                                        // the workspace is set up
};

struct ddp_sync_norm {
    int32_t world = 0, n_params = 0, n_buckets = 0, dtype = 0, divisor = 0, algo = 0;
    // the arguments of ddp_sync_buckets
    std::vector<void*> grads, buckets;
    std::vector<int64_t> numel, offset, bucket_numel;
    std::vector<int32_t> bucket_of;
    std::shared_ptr<const SyncPlan> sync;                      // the view algorithms' tables
    char* sync_table = nullptr;
    bool sync_ready = false;                                   // the workspace is set up for `sync`
    // rank 0's gradients, for a norm pass after a sync without one
    std::shared_ptr<const RangePlan> plan;
    std::vector<std::pair<uintptr_t, uintptr_t>> spans;        // the gradients and the workspace, sorted
    std::vector<std::pair<uintptr_t, uintptr_t>> bucket_spans; // the memory of the buckets, sorted and disjoint
    NormSpace space{nullptr, nullptr, nullptr};
    bool ready = false;                                        // the workspace is set up
};

struct ddp_adamw {
    int32_t world = 0, grad_dtype = 0;
    bool copies = false;
    std::shared_ptr<const AdamWPlan> plan;
    std::vector<std::pair<uintptr_t, uintptr_t>> spans;        // what a step writes, sorted
    int32_t* steps = nullptr;
    int32_t* arrivals = nullptr;
    char* table = nullptr;
    bool ready = false;                                        // the workspace is set up
};

namespace {

using Span = std::pair<uintptr_t, uintptr_t>;      // [first, second) in bytes

Span span_of(const void* p, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Span{a, a + (uintptr_t)bytes};
}

// Sorts the spans; true if two of them share a byte.
bool any_overlap(std::vector<Span>* v) {
    std::sort(v->begin(), v->end());
    for (size_t i = 1; i < v->size(); ++i)
        if ((*v)[i].first < (*v)[i - 1].second) return true;
    return false;
}

// Sorts the spans and joins those that share a byte or touch.
void unite(std::vector<Span>* v) {
    std::sort(v->begin(), v->end());
    size_t n = 0;
    for (const Span& s : *v) {
        if (n > 0 && s.first <= (*v)[n - 1].second) (*v)[n - 1].second = std::max((*v)[n - 1].second, s.second);
        else (*v)[n++] = s;
    }
    v->resize(n);
}

// True if s shares a byte with one of the sorted, disjoint spans.
bool hits_any(const std::vector<Span>& sorted, Span s) {
    auto it = std::lower_bound(sorted.begin(), sorted.end(), Span{s.second, 0});
    return it != sorted.begin() && std::prev(it)->second > s.first;
}

// World, tensor count and sizes shared by the creating calls.  A rank's
// elements are capped as one buffer's are, so that sums of bytes and tiles fit.
int32_t check_sizes(int32_t world, int32_t n_params, const int64_t* numel, int32_t dtype) {
    const int32_t st = common_checks(world, 0, dtype);
    if (st) return st;
    if (n_params < 0 || (n_params > 0 && !numel)) return DDP_ERR_INVALID;
    int64_t total = 0;
    for (int32_t i = 0; i < n_params; ++i) {
        const int32_t s = common_checks(world, numel[i], dtype);
        if (s) return s;
        total += numel[i];
        if (total > DDP_MAX_NUMEL) return DDP_ERR_CAPACITY;
    }
    return DDP_OK;
}

int32_t check_ptr(const void* p, int64_t align) {
    if (!p) return DDP_ERR_INVALID;
    return reinterpret_cast<uintptr_t>(p) % (uintptr_t)align ? DDP_ERR_ALIGN : DDP_OK;
}

// Appends tensor (p, bytes) of rank r, joined to the range before it where it continues it.
void add_range(std::vector<GradRange>* v, void* p, int64_t bytes, int32_t r) {
    char* c = static_cast<char*>(p);
    if (!v->empty() && v->back().rank == r && v->back().ptr + v->back().bytes == c) v->back().bytes += bytes;
    else v->push_back(GradRange{c, bytes, r});
}

// The most tiles that tensors of these sizes can take, wherever they lie; their
// partials are fewer, but for the padding of a rank's or a table's last run.
int64_t most_tiles(int32_t n_params, const int64_t* numel, int64_t es) {
    int64_t t = 0;
    for (int32_t i = 0; i < n_params; ++i)
        if (numel[i] > 0) t += (numel[i] * es + kNormAlign - 1) / kNormTile + 2;
    return t;
}

// Vectors a thread of the sync with norm takes.
int sync_vecs(int32_t world, int32_t n_params, const int64_t* numel, int32_t dtype) {
    int64_t n = 0;
    for (int32_t i = 0; i < n_params; ++i) n += numel[i];
    return sync_norm_vecs(world, n, dtype);
}

// `partials` is how many the workspace has room for; the table comes after them.
NormSpace space_of(void* workspace, int64_t partials) {
    char* w = static_cast<char*>(workspace);
    return NormSpace{reinterpret_cast<uint32_t*>(w), reinterpret_cast<double*>(w + kNormSpaceHead),
                     w + table_offset(kNormSpaceHead + 8 * partials)};
}

// Before the first launch that uses them: a handle's counter is zeroed and its
// table, if it is in device memory, written.  A capture records both for its
// replays, and proves nothing for later calls.
cudaError_t make_ready(void* counter, const DeviceTable* table, void* at, bool* ready, cudaStream_t stream) {
    if (*ready) return cudaSuccess;
    cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(stream, &capturing);
    if (e == cudaSuccess) e = cudaMemsetAsync(counter, 0, 4, stream);
    if (e == cudaSuccess && table) e = upload_table(*table, at, stream);
    if (e == cudaSuccess && capturing == cudaStreamCaptureStatusNone) *ready = true;
    return e;
}

int32_t ready(ddp_grad_set* s, cudaStream_t q) {
    return cuda_status(make_ready(s->space.counter, range_plan_table(*s->plan), s->space.table, &s->ready, q));
}

// The workspace of a sync with norm, the partials it has room for, and where the
// members' table goes (the ranges' comes right after the partials).
int32_t sync_norm_space(int32_t world, int32_t n_params, const int64_t* numel, int32_t dtype, int64_t* bytes,
                        int64_t* partials, int64_t* sync_table) {
    if (!bytes) return DDP_ERR_INVALID;
    const int32_t st = check_sizes(world, n_params, numel, dtype);
    if (st) return st;
    const int64_t tile = (int64_t)kThreads * sync_vecs(world, n_params, numel, dtype) * (16 / elem_bytes(dtype));
    int64_t tiles = 0;
    for (int32_t i = 0; i < n_params; ++i)
        if (numel[i] > 0) tiles += numel[i] / tile + 2;
    tiles = std::max(tiles, most_tiles(n_params, numel, elem_bytes(dtype)));
    if (partials) *partials = tiles;
    // members with their pointers, and ranges for a norm pass: which of them a run
    // needs can change from run to run, and a captured graph keeps its own
    const int64_t ranges = table_space(kNormSpaceHead + 8 * tiles, n_params, kRangeEntry);
    if (sync_table) *sync_table = table_offset(ranges);
    *bytes = table_space(ranges, n_params, kSyncEntry + 8 * (int64_t)world);
    return DDP_OK;
}

bool bad_max_norm(double max_norm) { return !(max_norm > 0.0) || !((float)max_norm > 0.f); }

}  // namespace

extern "C" {

int32_t ddp_grad_set_workspace_bytes(int32_t world, int32_t n_params, const int64_t* numel, int32_t dtype,
                                     int64_t* bytes) try {
    DDP_TRACE_CALL();
    if (!bytes) return DDP_ERR_INVALID;
    const int32_t st = check_sizes(world, n_params, numel, dtype);
    if (st) return st;
    *bytes = table_space(kNormSpaceHead + 8 * world * most_tiles(n_params, numel, elem_bytes(dtype)),
                         (int64_t)world * n_params, kRangeEntry);
    return DDP_OK;
} DDP_ABI_CATCH

int32_t ddp_grad_set_create(int32_t world, int32_t n_params, void* const* grads, const int64_t* numel, int32_t dtype,
                            void* workspace, int64_t workspace_bytes, ddp_grad_set** out) try {
    DDP_TRACE_CALL();
    if (!out) return DDP_ERR_INVALID;
    *out = nullptr;
    int64_t need = 0;
    int32_t st = ddp_grad_set_workspace_bytes(world, n_params, numel, dtype, &need);
    if (st) return st;
    if (n_params > 0 && !grads) return DDP_ERR_INVALID;
    if ((st = check_ptr(workspace, 16))) return st;
    if (workspace_bytes < need) return DDP_ERR_CAPACITY;
    if (need / 8 > INT32_MAX / 8) return DDP_ERR_CAPACITY;
    const int64_t es = elem_bytes(dtype);
    std::unique_ptr<ddp_grad_set> s(new ddp_grad_set());
    s->world = world;
    s->dtype = dtype;
    s->space = space_of(workspace, world * most_tiles(n_params, numel, es));
    s->spans.push_back(span_of(workspace, need));
    std::vector<GradRange> ranges;               // by rank, then by address
    std::vector<Span> rank;
    for (int32_t r = 0; r < world; ++r) {
        rank.clear();
        for (int32_t i = 0; i < n_params; ++i) {
            if (numel[i] == 0) continue;
            const void* g = grads[(int64_t)r * n_params + i];
            if ((st = check_ptr(g, es))) return st;
            rank.push_back(span_of(g, numel[i] * es));
        }
        std::sort(rank.begin(), rank.end());
        s->spans.insert(s->spans.end(), rank.begin(), rank.end());
        for (const Span& g : rank)
            add_range(&ranges, reinterpret_cast<void*>(g.first), (int64_t)(g.second - g.first), r);
    }
    s->plan = make_range_plan(ranges.data(), (int64_t)ranges.size(), world);
    if (any_overlap(&s->spans)) return DDP_ERR_INVALID;
    *out = s.release();
    return DDP_OK;
} DDP_ABI_CATCH

int32_t ddp_grad_norm(ddp_grad_set* s, float* norms, void* stream) try {
    DDP_TRACE_CALL();
    if (!s) return DDP_ERR_INVALID;
    int32_t st = check_ptr(norms, 4);
    if (st) return st;
    if (hits_any(s->spans, span_of(norms, 4 * (int64_t)s->world))) return DDP_ERR_INVALID;
    cudaStream_t q = (cudaStream_t)stream;
    if ((st = ready(s, q))) return st;
    return cuda_status(launch_norm(*s->plan, s->dtype, s->space, 1, norms, q));
} DDP_ABI_CATCH

int32_t ddp_grad_clip(ddp_grad_set* s, const float* norms, double max_norm, void* stream) try {
    DDP_TRACE_CALL();
    if (!s || bad_max_norm(max_norm)) return DDP_ERR_INVALID;
    int32_t st = check_ptr(norms, 4);
    if (st) return st;
    if (hits_any(s->spans, span_of(norms, 4 * (int64_t)s->world))) return DDP_ERR_INVALID;
    if ((st = ready(s, (cudaStream_t)stream))) return st;
    return cuda_status(launch_clip(*s->plan, s->dtype, s->space, norms, (float)max_norm, (cudaStream_t)stream));
} DDP_ABI_CATCH

int32_t ddp_grad_norm_clip(ddp_grad_set* s, float* norms, double max_norm, void* stream) try {
    DDP_TRACE_CALL();
    if (!s || bad_max_norm(max_norm)) return DDP_ERR_INVALID;
    const int32_t st = ddp_grad_norm(s, norms, stream);
    return st ? st : ddp_grad_clip(s, norms, max_norm, stream);
} DDP_ABI_CATCH

int32_t ddp_grad_set_destroy(ddp_grad_set* s) try {
    DDP_TRACE_CALL();
    delete s;
    return DDP_OK;
} DDP_ABI_CATCH

int32_t ddp_sync_norm_workspace_bytes(int32_t world, int32_t n_params, const int64_t* numel, int32_t dtype,
                                      int64_t* bytes) try {
    DDP_TRACE_CALL();
    return sync_norm_space(world, n_params, numel, dtype, bytes, nullptr, nullptr);
} DDP_ABI_CATCH

int32_t ddp_sync_norm_create(int32_t world, int32_t n_params, void* const* grads, const int64_t* numel,
                             const int32_t* bucket_of_param, const int64_t* offset_of_param, int32_t n_buckets,
                             const int64_t* bucket_numel, void* const* buckets, int32_t dtype, int32_t divisor,
                             int32_t algo, void* workspace, int64_t workspace_bytes, ddp_sync_norm** out) try {
    DDP_TRACE_CALL();
    if (!out) return DDP_ERR_INVALID;
    *out = nullptr;
    int64_t need = 0, partials = 0, sync_table = 0;
    int32_t st = sync_norm_space(world, n_params, numel, dtype, &need, &partials, &sync_table);
    if (st) return st;
    if (n_buckets < 0 || divisor < 0) return DDP_ERR_INVALID;
    const bool hook = algo == DDP_ALGO_BF16_HOOK || algo == DDP_ALGO_BF16_HOOK_VIEW || algo == DDP_ALGO_FP16_HOOK_VIEW;
    const bool needs_buckets = algo == DDP_ALGO_FUSED || algo == DDP_ALGO_STAGED || algo == DDP_ALGO_BF16_HOOK;
    if (!hook && !needs_buckets && algo != DDP_ALGO_VIEW) return DDP_ERR_INVALID;
    if (hook && dtype != DDP_F32) return DDP_ERR_INVALID;
    if (n_params > 0 && (!grads || !bucket_of_param || !offset_of_param)) return DDP_ERR_INVALID;
    if (n_buckets > 0 && (!bucket_numel || (needs_buckets && !buckets))) return DDP_ERR_INVALID;
    if ((st = check_ptr(workspace, 16))) return st;
    if (workspace_bytes < need || need / 8 > INT32_MAX / 8) return DDP_ERR_CAPACITY;
    for (int32_t k = 0; k < n_buckets; ++k)
        if ((st = common_checks(world, bucket_numel[k], dtype))) return st;
    std::unique_ptr<ddp_sync_norm> s(new ddp_sync_norm());
    s->world = world;
    s->n_params = n_params;
    s->n_buckets = n_buckets;
    s->dtype = dtype;
    s->divisor = divisor;
    s->algo = algo;
    s->space = space_of(workspace, partials);
    s->sync_table = static_cast<char*>(workspace) + sync_table;
    const int64_t all = (int64_t)world * n_params, es = elem_bytes(dtype);
    if (n_params > 0) {
        s->grads.assign(grads, grads + all);
        s->numel.assign(numel, numel + n_params);
        s->bucket_of.assign(bucket_of_param, bucket_of_param + n_params);
        s->offset.assign(offset_of_param, offset_of_param + n_params);
    }
    if (n_buckets > 0) s->bucket_numel.assign(bucket_numel, bucket_numel + n_buckets);
    // the plan: members inside their buckets, in offset order, disjoint
    std::vector<int32_t> order;
    for (int32_t p = 0; p < n_params; ++p) {
        const int32_t k = bucket_of_param[p];
        if (k < 0 || k >= n_buckets) return DDP_ERR_INVALID;
        if (offset_of_param[p] < 0 || offset_of_param[p] > bucket_numel[k] - numel[p]) return DDP_ERR_INVALID;
        if (numel[p] > 0) order.push_back(p);
    }
    std::sort(order.begin(), order.end(), [&](int32_t a, int32_t b) {
        return bucket_of_param[a] != bucket_of_param[b] ? bucket_of_param[a] < bucket_of_param[b]
                                                        : offset_of_param[a] < offset_of_param[b];
    });
    for (size_t i = 1; i < order.size(); ++i) {
        const int32_t a = order[i - 1], b = order[i];
        if (bucket_of_param[a] == bucket_of_param[b] && offset_of_param[a] + numel[a] > offset_of_param[b])
            return DDP_ERR_INVALID;
    }
    // the memory
    s->spans.push_back(span_of(workspace, need));
    for (int64_t k = 0; k < all; ++k) {
        const int64_t n = numel[k % n_params];
        if (n == 0) continue;
        if ((st = check_ptr(grads[k], es))) return st;
        s->spans.push_back(span_of(grads[k], n * es));
    }
    if (any_overlap(&s->spans)) return DDP_ERR_INVALID;
    if (needs_buckets && n_buckets > 0) {        // buckets may share memory with each other across k
        s->buckets.assign(buckets, buckets + (int64_t)world * n_buckets);
        const int64_t bs = algo == DDP_ALGO_BF16_HOOK ? 2 : es;
        for (int64_t k = 0; k < (int64_t)world * n_buckets; ++k) {
            const int64_t n = bucket_numel[k % n_buckets];
            if (n == 0) continue;
            if ((st = check_ptr(buckets[k], bs))) return st;
            if (hits_any(s->spans, span_of(buckets[k], n * bs))) return DDP_ERR_INVALID;
            s->bucket_spans.push_back(span_of(buckets[k], n * bs));
        }
        unite(&s->bucket_spans);
    }
    // a member that continues the one before it, in its bucket and at every rank, joins it
    std::vector<SyncMember> members;
    std::vector<void*> ptrs;
    ptrs.reserve(order.size() * (size_t)world);
    int32_t bucket = -1;
    for (int32_t p : order) {
        const int32_t k = bucket_of_param[p];
        SyncMember* m = bucket == k ? &members.back() : nullptr;
        bool joins = m && m->offset + m->numel == offset_of_param[p];
        for (int32_t r = 0; joins && r < world; ++r)
            joins = static_cast<char*>(m->ptrs[r]) + m->numel * es == grads[(int64_t)r * n_params + p];
        bucket = k;
        if (joins) {
            m->numel += numel[p];
            continue;
        }
        void* const* at = ptrs.data() + ptrs.size();
        for (int32_t r = 0; r < world; ++r) ptrs.push_back(grads[(int64_t)r * n_params + p]);
        members.push_back(SyncMember{numel[p], offset_of_param[p], chunk_len(bucket_numel[k], world), at});
    }
    const int launch_dtype = algo == DDP_ALGO_BF16_HOOK_VIEW   ? kDtypeHook
                             : algo == DDP_ALGO_FP16_HOOK_VIEW ? kDtypeHook16
                                                               : dtype;
    if (!needs_buckets)
        s->sync = make_sync_plan(world, members.data(), (int64_t)members.size(), sync_vecs(world, n_params, numel, dtype),
                                 launch_dtype, make_div(divisor));
    // every rank holds the same average after the sync: rank 0's norm is everybody's
    std::vector<GradRange> ranges;
    for (int32_t p = 0; p < n_params; ++p)
        if (numel[p] > 0) add_range(&ranges, grads[p], numel[p] * es, 0);
    s->plan = make_range_plan(ranges.data(), (int64_t)ranges.size(), 1);
    *out = s.release();
    return DDP_OK;
} DDP_ABI_CATCH

int32_t ddp_sync_norm_run(ddp_sync_norm* s, float* norms, void* stream) try {
    DDP_TRACE_CALL();
    if (!s) return DDP_ERR_INVALID;
    int32_t st = check_ptr(norms, 4);
    if (st) return st;
    const Span out = span_of(norms, 4 * (int64_t)s->world);
    if (hits_any(s->spans, out) || hits_any(s->bucket_spans, out)) return DDP_ERR_INVALID;
    cudaStream_t q = (cudaStream_t)stream;
    // the kernel with the norm is a register kernel: where the TMA-staged view
    // kernel is asked for, or the CTA budget is one that it needs, the sync
    // runs as ddp_sync_buckets runs it and the norm takes a pass over rank 0.
    // From 16 ranks, below 128 MiB moved, ddp_sync_buckets takes the TMA-staged
    // kernel by itself; this call stays on its own there, which wins and loses
    // (this call, then sync and norm pass, in us): 16 ranks of 1.26M elements in
    // 184 tensors 36.2 and 43.1, of 500K in 40 19.0 and 17.6; 32 ranks of 30K in
    // 40 15.3 and 30.3, of 250K in 40 21.9 and 18.8; 64 ranks of 16K in 40 28.6
    // and 48.3, of 250K in 60 59.3 and 45.5
    const bool fused = s->sync && fused_kernel_override() != DDP_FUSED_TMA && !cta_cap_is_tight();
    if (fused) {
        NormSpace ws = s->space;
        ws.table = s->sync_table;
        if ((st = cuda_status(make_ready(ws.counter, sync_plan_table(*s->sync), ws.table, &s->sync_ready, q)))) return st;
        return cuda_status(launch_sync_norm(*s->sync, ws, norms, q));
    }
    if ((st = cuda_status(make_ready(s->space.counter, range_plan_table(*s->plan), s->space.table, &s->ready, q)))) return st;
    st = ddp_sync_buckets(s->world, s->n_params, s->grads.data(), s->numel.data(), s->bucket_of.data(), s->offset.data(),
                          s->n_buckets, s->bucket_numel.data(), s->buckets.empty() ? nullptr : s->buckets.data(), s->dtype,
                          s->divisor, s->algo, stream);
    if (st) return st;
    return cuda_status(launch_norm(*s->plan, s->dtype, s->space, s->world, norms, q));
} DDP_ABI_CATCH

int32_t ddp_sync_norm_destroy(ddp_sync_norm* s) try {
    DDP_TRACE_CALL();
    delete s;
    return DDP_OK;
} DDP_ABI_CATCH

int32_t ddp_adamw_workspace_bytes(int32_t world, int32_t n_params, int64_t* bytes) try {
    DDP_TRACE_CALL();
    const int32_t st = common_checks(world, 0, DDP_F32);
    if (st) return st;
    if (!bytes || n_params < 0) return DDP_ERR_INVALID;
    *bytes = table_space(kNormSpaceHead, (int64_t)world * n_params, kAdamWEntry);
    return DDP_OK;
} DDP_ABI_CATCH

int32_t ddp_adamw_create(int32_t world, int32_t n_params, void* const* params, const void* const* grads,
                         int32_t grad_dtype, void* const* exp_avg, void* const* exp_avg_sq, void* const* copies,
                         const int64_t* numel, const uint8_t* no_decay, int32_t* steps, void* workspace,
                         int64_t workspace_bytes, ddp_adamw** out) try {
    DDP_TRACE_CALL();
    if (!out) return DDP_ERR_INVALID;
    *out = nullptr;
    int32_t st = check_sizes(world, n_params, numel, grad_dtype);
    if (st) return st;
    if (n_params > 0 && (!params || !grads || !exp_avg || !exp_avg_sq)) return DDP_ERR_INVALID;
    if ((st = check_ptr(steps, 4)) || (st = check_ptr(workspace, 16))) return st;
    int64_t need = 0;
    if ((st = ddp_adamw_workspace_bytes(world, n_params, &need))) return st;
    if (workspace_bytes < need) return DDP_ERR_CAPACITY;
    std::unique_ptr<ddp_adamw> a(new ddp_adamw());
    a->world = world;
    a->grad_dtype = grad_dtype;
    a->copies = copies != nullptr;
    a->steps = steps;
    a->arrivals = static_cast<int32_t*>(workspace);
    a->table = static_cast<char*>(workspace) + table_offset(kNormSpaceHead);
    a->spans.push_back(span_of(steps, 4 * (int64_t)world));
    a->spans.push_back(span_of(workspace, need));
    std::vector<Span> read;
    const int64_t gs = elem_bytes(grad_dtype);
    std::vector<AdamWItem> items;
    int64_t tiles = 0;
    for (int32_t r = 0; r < world; ++r)
        for (int32_t i = 0; i < n_params; ++i) {
            if (numel[i] == 0) continue;
            const int64_t k = (int64_t)r * n_params + i;
            AdamWItem it{static_cast<float*>(params[k]),
                         static_cast<float*>(exp_avg[k]),
                         static_cast<float*>(exp_avg_sq[k]),
                         grads[k],
                         copies ? copies[k] : nullptr,
                         numel[i],
                         r,
                         no_decay && no_decay[i] ? 0 : 1};
            if ((st = check_ptr(it.p, 4)) || (st = check_ptr(it.m, 4)) || (st = check_ptr(it.v, 4)) ||
                (st = check_ptr(it.g, gs)) || (copies && (st = check_ptr(it.copy, 2))))
                return st;
            for (const void* p : {(const void*)it.p, (const void*)it.m, (const void*)it.v})
                a->spans.push_back(span_of(p, 4 * it.numel));
            if (copies) a->spans.push_back(span_of(it.copy, 2 * it.numel));
            read.push_back(span_of(it.g, gs * it.numel));
            // a tensor that continues the one before it in every array joins it
            AdamWItem* b = items.empty() ? nullptr : &items.back();
            if (b && b->rank == r && b->decay == it.decay && b->p + b->numel == it.p && b->m + b->numel == it.m &&
                b->v + b->numel == it.v && static_cast<const char*>(b->g) + gs * b->numel == it.g &&
                (!copies || static_cast<char*>(b->copy) + 2 * b->numel == it.copy))
                b->numel += it.numel;
            else
                items.push_back(it);
        }
    for (const AdamWItem& it : items) tiles += adamw_tiles(it);
    if (tiles > INT32_MAX / 8) return DDP_ERR_CAPACITY;
    if (any_overlap(&a->spans)) return DDP_ERR_INVALID;
    for (const Span& g : read)
        if (hits_any(a->spans, g)) return DDP_ERR_INVALID;
    a->plan = make_adamw_plan(items.data(), (int64_t)items.size(), grad_dtype, a->copies);
    *out = a.release();
    return DDP_OK;
} DDP_ABI_CATCH

int32_t ddp_adamw_step(ddp_adamw* a, double lr, double beta1, double beta2, double eps, double weight_decay,
                       const float* norms, double max_norm, void* stream) try {
    DDP_TRACE_CALL();
    if (!a) return DDP_ERR_INVALID;
    if (!(lr >= 0.0) || !std::isfinite(lr) || !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) ||
        !((float)eps > 0.f) || !std::isfinite(eps) || !(weight_decay >= 0.0) || !std::isfinite(weight_decay))
        return DDP_ERR_INVALID;
    if (norms) {
        if (bad_max_norm(max_norm)) return DDP_ERR_INVALID;
        const int32_t st = check_ptr(norms, 4);
        if (st) return st;
        if (hits_any(a->spans, span_of(norms, 4 * (int64_t)a->world))) return DDP_ERR_INVALID;
    }
    const int32_t st = cuda_status(make_ready(a->arrivals, adamw_plan_table(*a->plan), a->table, &a->ready,
                                              (cudaStream_t)stream));
    if (st) return st;
    const AdamWScalars s{(float)lr,
                         (float)beta1,
                         (float)(1.0 - beta1),
                         (float)std::log(beta1),
                         (float)beta2,
                         (float)(1.0 - beta2),
                         (float)std::log(beta2),
                         (float)eps,
                         (float)(lr * weight_decay),
                         (float)max_norm};
    return cuda_status(launch_adamw(*a->plan, a->table, a->world, a->grad_dtype, a->copies, s, norms, a->steps, a->arrivals,
                                    (cudaStream_t)stream));
} DDP_ABI_CATCH

int32_t ddp_adamw_destroy(ddp_adamw* a) try {
    DDP_TRACE_CALL();
    delete a;
    return DDP_OK;
} DDP_ABI_CATCH

}  // extern "C"
