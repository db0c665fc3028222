// loss_gemm.cu -- the loss head's matrix products on the fifth-generation tensor
// cores, with the softmax in their epilogues.
//
// With h the rows of learned tokens [T, d], w the weights [V, d] and dz the
// logits' gradients of one piece of the vocabulary [T, Vp]:
//   kStats     z = h w^T, never stored: every tile of 128 x 256 logits leaves a
//              maximum and a sum of exponentials for each row and 128 columns,
//              and the logits at the columns that a row lists;
//   kKeep      the same, and the exponentials themselves in 16 bits, where those of
//              all columns have room; a pass of its own makes dz of them;
//   kGrad      where they have not: z again, piece by piece, and
//              dz = softmax(z) - target, bf16;
//   kProducts  dh += dz w (over the piece's columns) and dw = f dz^T h (over T).
// The factor f (scale and reduction) stays out of dz: a target's dz lies just above -1, where bf16 is off by 2^-9 of it at
// most; times an arbitrary f it could be off by twice that, and by the same in every row.
// Both operands of kProducts are read as they lie in memory: the tensor cores
// take matrices whose rows run along the depth or across it.
//
// One block an SM walks over tiles.  A thread issues the tiles' loads (TMA, one an
// operand and stage of a ring in shared memory), another the products
// (tcgen05.mma, accumulators in tensor memory, two tiles' worth), eight warps
// take finished tiles out of tensor memory while the next one is computed.
//
// float32 operands are three bf16 planes, x = x0 + x1 + x2 (8 bits of the
// significand each); of the nine products of planes the six larger are summed,
// smallest first: what is left out is below 2^-24 of the terms.
//
// Bound by the tensor cores and, in calls after one another, by power: 8 x 1024 tokens by 50257 x 1024 take 0.55 ms for the
// logits and 1.03 ms for the products by themselves (1.52 and 1.64 PFLOP/s), 4096 by 131072 x 4096 2.37 and 4.78 ms (1.85
// and 1.84), in a row 2.61 and 5.48 (1.69 and 1.60).  Tiles are as large as two of them fit tensor memory: 128 x 256.
//
// Waits for loads, products, tiles and accumulators are bounded: one that runs
// out sets DDP_ERR_TIMEOUT in the device status word, the block's roles stop,
// loads in flight and products are waited for, and tensor memory is freed.  What
// waits without a limit waits for nothing that can fail to come: a barrier of the
// block or of a group's four warps, which all of them reach whatever has run out;
// the copy engine's own stores; and tensor memory at the start, which no other
// block of this kernel holds, for its shared memory leaves room for one an SM.
// No block waits for another one.  Pairs of SMs on one tile (cta_group::2) did,
// and were up to a tenth faster on large batches, but a float32 call in pairs
// once did not finish and no cause was found.
#include <algorithm>
#include <mutex>
#include <set>
#include <utility>

#include "ddp_device.cuh"
#include "loss_internal.h"

namespace ddpk {
namespace {

constexpr int kStages = 4;
constexpr int kBytesA = kTileM * kTileK * 2, kBytesB = kTileN * kTileK * 2, kBytesStage = kBytesA + kBytesB;
constexpr int kBytesBox = 64 * 64 * 2;
constexpr int kBytesStaging = 128 * 128;               // 128 rows of 128 bytes
constexpr int kFirstEpilogueWarp = 4, kEpilogueWarps = 8;
constexpr int kGemmThreads = 32 * (kFirstEpilogueWarp + kEpilogueWarps);
constexpr float kKeepScale = (float)(1 << kKeepBits);

// A tile: rank (-1: no more tiles), first row (of all ranks' rows; a column of the piece for dw), first column, columns (of
// the products: a multiple of 64), k blocks.
struct alignas(16) Tile {
    int32_t rank, m, n, columns, k0, k1, split;
    int32_t flags;
    __device__ __forceinline__ bool weights() const { return flags & 1; }      // of dw
    __device__ __forceinline__ bool more() const { return flags & 2; }         // added to the depth before
    __device__ __forceinline__ bool stalls() const { return flags & 4; }       // where a planted stall begins
};
// float32 sums are taken out of tensor memory and added up elsewhere every so many k blocks: the tensor cores cut what they
// add to a long sum (kCutPerStep), by 2e-5 of the result over a depth of 50257.
constexpr int kMostDepth = 16;
constexpr int kQueue = 4;

struct Control {
    Tile queue[kQueue];
    uint64_t full[kStages], empty[kStages];
    uint64_t ready[2], taken[2];                       // accumulators
    uint64_t tile_full[kQueue], tile_empty[kQueue];
    uint64_t drain;
    uint32_t tmem;
    int32_t stop;
    int32_t go[2][2];                                  // by group and accumulators: the tile is there
    int32_t counts[kLossRanks];
    float factors[kLossRanks];
};
constexpr int kSmem = 1024 + kStages * kBytesStage + 2 * kBytesStaging + (int)sizeof(Control);
static_assert(kSmem <= 227 * 1024, "shared memory of a block");
static_assert(2 * kSmem > 228 * 1024, "one block an SM: each takes all tensor memory");

__device__ __forceinline__ uint32_t smem_of(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void bar_init(uint64_t* b, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_of(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_of(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_of(b)) : "memory");
}
__device__ __forceinline__ void warp_arrive(uint64_t* b, int lane) {
    __syncwarp();
    if (lane == 0) bar_arrive(b);
}
__device__ __forceinline__ bool bar_try(uint64_t* b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_of(b)), "r"(parity)
        : "memory");
    return ok != 0;
}
// Whether the phase is complete, at once.
__device__ __forceinline__ bool bar_test(uint64_t* b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_of(b)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ unsigned long long now_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// At most limit_ns, or until another role of the block has given up; false then.
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, Control* s, const LossGemm& g) {
    if (bar_try(b, parity)) return true;
    const unsigned long long t0 = now_ns();
    while (!bar_try(b, parity)) {
        if (*(volatile int32_t*)&s->stop) return false;
        if (now_ns() - t0 > g.limit_ns) {
            *(volatile int32_t*)&s->stop = 1;
            atomicExch(g.c.status, DDP_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}
// The same after a role has given up: for what is still in flight.
__device__ __forceinline__ void bar_wait_rest(uint64_t* b, uint32_t parity, const LossGemm& g) {
    const unsigned long long t0 = now_ns();
    while (!bar_try(b, parity))
        if (now_ns() - t0 > g.limit_ns) return;
}

// A box of a matrix seen as [planes][columns / 64][rows][64], from column x (a multiple of 64) and row y.
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y, int plane, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(smem_of(dst)), "l"(map), "r"(0), "r"(y), "r"(x / 64), "r"(plane), "r"(smem_of(bar))
        : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
                 "r"(smem_of(src)), "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void tma_add_2d(const CUtensorMap* map, const void* src, int x, int y) {
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
                 "r"(smem_of(src)), "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void tma_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void tma_read_done() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_all_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void to_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A group's four warps meet, each of them whole: one lane may come from work of its own.
__device__ __forceinline__ void group_sync(int group) {
    __syncwarp();
    asm volatile("bar.sync %0, 128;" ::"r"(group + 1) : "memory");
}

// Shared-memory matrix descriptor: 128-byte swizzle, groups of 8 rows of 128 bytes
// 1024 bytes apart; lbo: bytes between runs of 64 elements across the depth.
__device__ __forceinline__ uint64_t matrix_desc(uint32_t addr, uint32_t lbo) {
    return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Instruction descriptor: bf16 x bf16 into float32, m x n; `across`: rows run across the depth.
__device__ __forceinline__ uint32_t product_desc(bool a_across, bool b_across, int m, int n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_across ? 1u : 0u) << 15) | ((b_across ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(desc), "r"((uint32_t)add)
        : "memory");
}
// The products issued so far arrive at the barrier.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_of(bar)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tmem_load(float* v, uint32_t addr) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    __syncwarp();                          // the load takes the whole warp
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// 2^x by the special-function unit: off by 2^-22 of the value at most, 0 below 2^-126.
__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two floats at a time.
struct Pair {
    uint64_t bits;
    __device__ __forceinline__ Pair(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(bits) : "f"(a), "f"(b)); }
    __device__ __forceinline__ explicit Pair(uint64_t x) : bits(x) {}
    __device__ __forceinline__ float2 get() const {
        float2 v;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(bits));
        return v;
    }
};
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a.bits), "l"(b.bits));
    return Pair(r);
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a.bits), "l"(b.bits));
    return Pair(r);
}
__device__ __forceinline__ Pair exp2_of(Pair x) {
    const float2 v = x.get();
    return Pair(exp2_of(v.x), exp2_of(v.y));
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Tiles of rank i in the phase: of its rows first, of its weights' gradients behind those of all ranks.
template <LossPhase PHASE>
__device__ __forceinline__ int phase_columns(const LossGemm& g) {
    return PHASE == LossPhase::kProducts ? g.c.dim : PHASE == LossPhase::kGrad ? g.width : g.c.vocab;
}
template <LossPhase PHASE>
__device__ __forceinline__ bool find_tile(const LossGemm& g, const int32_t* counts, int t, Tile* w) {
    const int all = phase_columns<PHASE>(g), nt = ceil_div(all, kTileN);
    for (int i = 0; i < g.n; ++i) {
        const int m = ceil_div(counts[i], kTileM), n = m * nt * (PHASE == LossPhase::kProducts ? g.splits : 1);
        if (t >= n) {
            t -= n;
            continue;
        }
        w->rank = i;
        w->flags = 0;
        w->split = 0;
        if (PHASE != LossPhase::kProducts) {           // rows' tiles of one column block together: they share the weights
            w->m = g.row0[i] + t % m * kTileM;
            w->n = t / m * kTileN;
            w->k0 = 0;
            w->k1 = g.c.dimp / kTileK;
        } else {
            w->n = t % nt * kTileN;
            t /= nt;
            w->m = g.row0[i] + t % m * kTileM;
            w->split = t / m;
            w->k0 = w->split * g.split_blocks;
            w->k1 = min(w->k0 + g.split_blocks, ceil_div(g.width, kTileK));
        }
        w->columns = ceil_div(min(all - w->n, kTileN), 64) * 64;
        return true;
    }
    if constexpr (PHASE == LossPhase::kProducts) {
        for (int i = 0; i < g.n; ++i) {
            const int n = counts[i] == 0 && g.accumulate ? 0 : ceil_div(g.width, kTileM) * nt;
            if (t >= n) {
                t -= n;
                continue;
            }
            w->rank = i;
            w->flags = 1;
            w->split = 0;
            w->n = t % nt * kTileN;
            w->m = t / nt * kTileM;
            w->k0 = 0;
            w->k1 = ceil_div(counts[i], kTileK);
            w->columns = ceil_div(min(all - w->n, kTileN), 64) * 64;
            return true;
        }
    }
    return false;
}

__device__ __forceinline__ void put_tile(Tile* at, const Tile& w) {
    static_assert(sizeof(Tile) == 32, "two vectors");
    const int32_t* from = reinterpret_cast<const int32_t*>(&w);
#pragma unroll
    for (int i = 0; i < 8; i += 4)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(smem_of(at) + 4 * i), "r"(from[i]), "r"(from[i + 1]),
                     "r"(from[i + 2]), "r"(from[i + 3])
                     : "memory");
}
__device__ __forceinline__ void get_tile(Tile* w, const Tile* at) {
    int32_t* to = reinterpret_cast<int32_t*>(w);
#pragma unroll
    for (int i = 0; i < 8; i += 4)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(to[i]), "=r"(to[i + 1]), "=r"(to[i + 2]), "=r"(to[i + 3])
                     : "r"(smem_of(at) + 4 * i)
                     : "memory");
}

// ---- the tiles' queue -----------------------------------------------------------
// Tiles differ in depth, so blocks take them as they come: the first each by its number, the others from a counter in
// device memory.  A thread decodes them ahead of the other roles.  Who computes a tile changes no value.  The last block
// to finish leaves the counters at zero.
template <LossPhase PHASE, bool F32>
__device__ void schedule(const LossGemm& g, Control* s) {
    int slot = 0, t = blockIdx.x;
    uint32_t phase = 1;
    bool more = true;
    while (more) {
        Tile w;
        more = find_tile<PHASE>(g, s->counts, t, &w);
        if (more && t == g.stall) w.flags |= 4;
        if (more) t = (int)gridDim.x + atomicAdd(g.c.next, 1);
        else w.rank = -1;
        const int end = w.k1;
        do {                               // a tile's depth, in parts that follow each other
            if (F32 && PHASE == LossPhase::kProducts && more) w.k1 = min(end, w.k0 + kMostDepth);
            if (!bar_wait(&s->tile_empty[slot], phase, s, g)) {
                more = false;
                break;
            }
            put_tile(&s->queue[slot], w);
            bar_arrive(&s->tile_full[slot]);
            if (++slot == kQueue) {
                slot = 0;
                phase ^= 1;
            }
            w.k0 = w.k1;
            w.flags |= 2;
        } while (more && w.k1 < end);
    }
    __threadfence();
    if (atomicAdd(g.c.next + 1, 1) == (int)gridDim.x - 1) {
        g.c.next[0] = 0;
        g.c.next[1] = 0;
    }
}

// The place of a role in its block's queue.
struct Queue {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ bool wait(Control* s, const LossGemm& g) {
        return bar_wait(&s->tile_full[slot], phase, s, g);
    }
    __device__ __forceinline__ void read(Control* s, Tile* w) const { get_tile(w, &s->queue[slot]); }
    __device__ __forceinline__ void done(Control* s) {
        bar_arrive(&s->tile_empty[slot]);
        step();
    }
    __device__ __forceinline__ void step() {
        if (++slot == kQueue) {
            slot = 0;
            phase ^= 1;
        }
    }
    // For a role of one thread: the next tile; false at the end, or where the wait gave up (rank then is -2).
    __device__ __forceinline__ bool next(Control* s, const LossGemm& g, Tile* w) {
        if (!wait(s, g)) {
            w->rank = -2;
            return false;
        }
        read(s, w);
        done(s);
        return w->rank >= 0;
    }
};

// Who reads the queue: the loads, the products and the epilogue's warps.
constexpr int kQueueReaders = 2 + kEpilogueWarps;

__device__ constexpr int8_t kPlaneA[6] = {2, 1, 0, 1, 0, 0};
__device__ constexpr int8_t kPlaneB[6] = {0, 1, 2, 0, 1, 0};

// ---- producer -----------------------------------------------------------------
template <LossPhase PHASE, bool F32>
__device__ void produce(const LossGemm& g, Control* s, char* stages) {
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    Queue queue;
    Tile w;
    while (ok && queue.next(s, g, &w) && !w.stalls()) {
        const CUtensorMap* wmap = &g.weights[w.rank];
        for (int q = 0; ok && q < (F32 ? 6 : 1); ++q) {
            const int pa = F32 ? kPlaneA[q] : 0, pb = F32 ? kPlaneB[q] : 0;
            for (int kb = w.k0; kb < w.k1; ++kb) {
                if (!bar_wait(&s->empty[stage], phase ^ 1, s, g)) {
                    ok = false;
                    break;
                }
                char* a = stages + stage * kBytesStage;
                char* b = a + kBytesA;
                uint64_t* const bar = &s->full[stage];
                bar_expect(bar, kBytesStage);
                const int k = kb * kTileK;
                if (PHASE != LossPhase::kProducts) {
                    tma_load(a, &g.hidden, k, w.m, pa, bar);
                    tma_load(b, wmap, k, g.piece0 + w.n, pb, bar);
                } else if (!w.weights()) {
                    tma_load(a, &g.piece, k, w.m - g.row0[0], pa, bar);
                    tma_load(b, wmap, w.n, g.piece0 + k, pb, bar);
                } else {
                    const int row = g.row0[w.rank] + k;
                    tma_load(a, &g.piece_across, w.m, row - g.row0[0], pa, bar);
                    tma_load(b, &g.hidden, w.n, row, pb, bar);
                }
                ++issued;
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
    }
    ok = ok && w.rank == -1;
    // what the products still have to report arrives here before the block ends
    for (int i = 0; ok && i < kStages; ++i) {
        ok = bar_wait(&s->empty[stage], phase ^ 1, s, g);
        if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
        }
    }
    if (!ok)                               // loads in flight, before the block's shared memory goes
        for (int i = max(0, issued - kStages); i < issued; ++i) bar_wait_rest(&s->full[i % kStages], (i / kStages) & 1, g);
}

// ---- products -----------------------------------------------------------------
// The tensor cores' own queue is short: the next stage is looked up before a stage's last product is issued, and the next
// tile while the present one's are.
template <LossPhase PHASE, bool F32>
__device__ void multiply(const LossGemm& g, Control* s, char* stages, uint32_t tmem) {
    int stage = 0, buf = 0;
    uint32_t phase = 0, taken = 1;
    bool ok = true, there = false;
    Queue queue;
    Tile w, after;
    bool more = queue.next(s, g, &w);
    while (more) {
        const bool a_across = PHASE == LossPhase::kProducts && w.weights(), b_across = PHASE == LossPhase::kProducts;
        const uint32_t desc = product_desc(a_across, b_across, kTileM, w.columns);
        // 16 elements of depth: 32 bytes along a row, or 16 rows of 128 bytes
        const uint32_t step_a = a_across ? 16 * 128 / 16 : 2, step_b = b_across ? 16 * 128 / 16 : 2;
        if (!(ok = bar_wait(&s->taken[buf], taken, s, g))) break;
        fence_after();
        const int blocks = max(w.k1 - w.k0, 0) * (F32 ? 6 : 1);
        for (int i = 0; i < blocks; ++i) {
            if (!there && !(ok = bar_wait(&s->full[stage], phase, s, g))) break;
            fence_after();
            const uint32_t a = smem_of(stages + stage * kBytesStage);
            const uint64_t da = matrix_desc(a, kBytesBox), db = matrix_desc(a + kBytesA, kBytesBox);
            uint64_t* const empty = &s->empty[stage];
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1;
            }
#pragma unroll
            for (int k = 0; k < kTileK / 16; ++k) {
                if (k == kTileK / 16 - 1) there = bar_test(&s->full[stage], phase);
                mma(tmem + buf * kTileN, da + k * step_a, db + k * step_b, desc, i > 0 || k > 0);
            }
            mma_commit(empty);
            if (i == 0) more = queue.next(s, g, &after);
        }
        if (!ok) break;
        mma_commit(&s->ready[buf]);
        if (blocks == 0) more = queue.next(s, g, &after);
        if (buf == 1) taken ^= 1;
        buf ^= 1;
        w = after;
    }
    if (!ok || w.rank == -2) {             // products in flight, before tensor memory goes
        mma_commit(&s->drain);
        bar_wait_rest(&s->drain, 0, g);
    }
}

// ---- epilogues -----------------------------------------------------------------
// A thread has one row of the tile and 128 of its columns; `mine` is its row of
// the group's staging buffer (128 bytes), whose 16-byte pieces are permuted by `turn`.
struct Lane {
    int group, quarter, lane, row;         // row of the tile
    uint32_t tmem;                         // the row's columns of this group
    char* staging;                         // the group's
    char* mine;
    int turn;
    bool leader;                           // of the group's 128 threads
};

__device__ __forceinline__ void stage_floats(const Lane& l, const float* v) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        *reinterpret_cast<float4*>(l.mine + ((i ^ l.turn) << 4)) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}
__device__ __forceinline__ float staged_float(const Lane& l, int i) {
    return *reinterpret_cast<const float*>(l.mine + (((i >> 2) ^ l.turn) << 4) + (i & 3) * 4);
}

// The columns that a row lists within its group's columns, in order.
template <bool LIST>
struct Listed {
    int64_t at;                            // of the entry in the arrays [][list]
    int64_t end;
    int column;                            // of the entry; past every column where there is none
    const int32_t* columns;
    __device__ __forceinline__ void start(const LossCall& c, int row, int token, int first, bool valid) {
        columns = c.columns;
        if (LIST) {
            const uint16_t* s = c.starts + (int64_t)token * (c.units + 1) + first / kLossUnit;
            at = (int64_t)token * c.list;
            end = at + (valid ? s[1] : 0);
            at += valid ? s[0] : 0;
            column = at < end ? columns[at] : INT32_MAX;
        } else {
            at = row;
            column = valid ? c.row_column[row] : INT32_MAX;
            if (column < first || column >= first + kLossUnit) column = INT32_MAX;
        }
    }
    __device__ __forceinline__ void next() {
        ++at;
        column = LIST && at < end ? columns[at] : INT32_MAX;
    }
};

// Twice over the row's 128 logits: their maximum, and their exponentials relative to it, whose arguments are taken after
// the subtraction: the largest is 1 whatever the logits' size.  One of the ones stays out of the sum (LossCall::partial): it
// is taken off, or, of a sum below kConfident, whose rest would lack digits, left out in going over the logits again.
// KEEP: the exponentials are stored, for bf16 operands as binary16, 2^kKeepBits for the row's largest, so that those down
// to 2^-29 of it keep 11 bits, for float32 as they are.
constexpr float kConfident = 1.125f;                   // the rest is off by 9 steps of a sum at most

// The sum of the unit's exponentials but for the largest, which is there once.
__device__ __forceinline__ float rest_of(const Lane& l, float ref, float k, int columns) {
    float rest = 0.f;
#pragma unroll 1
    for (int j = 0; j < kLossUnit / 32; ++j) {
        float v[32];
        tmem_load(v, l.tmem + j * 32);
        tmem_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float d = v[i] - ref;
            if (j * 32 + i < columns && d != 0.f) rest += exp2_of(d * k);
        }
    }
    return rest;
}

template <bool F32, bool TWO, bool LIST, bool KEEP>
__device__ __forceinline__ void stats_tile(const LossGemm& g, const Tile& w, const Lane& l, Control* s, uint64_t* taken) {
    const LossCall& c = g.c;
    const int row = w.m + l.row, first = w.n + l.group * kLossUnit;
    const bool valid = row - g.row0[w.rank] < s->counts[w.rank];
    Listed<LIST> hit;
    hit.start(c, row, LIST && valid ? g.row0[w.rank] + c.row_token[row] : 0, first, valid && first < c.vocab);
    const float k1 = c.k1, k2 = c.k2;
    if (KEEP) {
        if (l.leader) tma_read_done();
        group_sync(l.group);               // the staging buffer is free
    }
    float top = -INFINITY;
#pragma unroll 1
    for (int j = 0; j < kLossUnit / 32; ++j) {
        float v[32];
        tmem_load(v, l.tmem + j * 32);
        tmem_wait();
        const int col = first + j * 32;
        if (__any_sync(0xffffffffu, hit.column < col + 32)) {
            stage_floats(l, v);
            while (hit.column < col + 32) {
                c.z[hit.at] = staged_float(l, hit.column - col);
                hit.next();
            }
        }
        if (col + 32 > c.vocab) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (col + i >= c.vocab) v[i] = -INFINITY;
        }
        float m[4] = {top, v[1], v[2], v[3]};
        m[0] = fmaxf(top, v[0]);
#pragma unroll
        for (int i = 4; i < 32; ++i) m[i & 3] = fmaxf(m[i & 3], v[i]);
        top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
    }
    const float ref = top == -INFINITY ? 0.f : top;    // nothing but -infinity: no terms
    const bool flat = TWO && k2 < k1;                  // the flatter softmax's exponentials are kept
    const Pair from(-ref, -ref), k1s(k1, k1), k2s(k2, k2);
    Pair sum[2] = {Pair(0.f, 0.f), Pair(0.f, 0.f)}, sum2[2] = {Pair(0.f, 0.f), Pair(0.f, 0.f)};
    float rest = 0.f, rest2 = 0.f;
    constexpr int kColumns = KEEP && !F32 ? 64 : 32;   // kept in 128 bytes
#pragma unroll 1
    for (int j = 0; j < kLossUnit / kColumns; ++j) {
        const int col = first + j * kColumns;
        uint32_t kept[32];
#pragma unroll
        for (int h = 0; h < kColumns / 32; ++h) {
            float v[32];
            tmem_load(v, l.tmem + j * kColumns + h * 32);
            tmem_wait();
            if (col + h * 32 + 32 > c.vocab) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (col + h * 32 + i >= c.vocab) v[i] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const Pair d = Pair(v[i], v[i + 1]) + from, x = exp2_of(d * k1s);
                sum[i / 2 & 1] = sum[i / 2 & 1] + x;
                float2 e = x.get();
                if (TWO) {
                    const Pair y = exp2_of(d * k2s);
                    sum2[i / 2 & 1] = sum2[i / 2 & 1] + y;
                    if (flat) e = y.get();
                }
                if (KEEP && F32) {
                    kept[i] = __float_as_uint(e.x);
                    kept[i + 1] = __float_as_uint(e.y);
                } else if (KEEP) {
                    const __half2 p = __floats2half2_rn(e.x * kKeepScale, e.y * kKeepScale);
                    kept[h * 16 + i / 2] = *reinterpret_cast<const uint32_t*>(&p);
                }
            }
        }
        if (j == kLossUnit / kColumns - 1) {
            const float2 a = (sum[0] + sum[1]).get(), b = (sum2[0] + sum2[1]).get();
            const float total = a.x + a.y, total2 = b.x + b.y;
            const bool some = top != -INFINITY;        // else no 1: 0, or NaN
            rest = some ? total - 1.f : total;
            rest2 = some ? total2 - 1.f : total2;
            const bool confident = valid && some && total < kConfident, confident2 = TWO && valid && some && total2 < kConfident;
            if (__any_sync(0xffffffffu, confident)) {
                const float r = rest_of(l, ref, k1, c.vocab - first);
                if (confident) rest = r;
            }
            if (TWO && __any_sync(0xffffffffu, confident2)) {
                const float r = rest_of(l, ref, k2, c.vocab - first);
                if (confident2) rest2 = r;
            }
            fence_before();
            warp_arrive(taken, l.lane);
        }
        if (KEEP) {
            if (j > 0) {
                if (l.leader) tma_read_done();
                group_sync(l.group);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                *reinterpret_cast<uint4*>(l.mine + ((i ^ l.turn) << 4)) =
                    make_uint4(kept[4 * i], kept[4 * i + 1], kept[4 * i + 2], kept[4 * i + 3]);
            to_async_proxy();
            group_sync(l.group);
            if (l.leader) {
                tma_store_2d(&g.keep_out, l.staging, w.n + l.group * kLossUnit + j * kColumns, w.m - g.row0[0]);
                tma_commit();
            }
        }
    }
    if (valid && first < c.vocab) {
        const int64_t at = (int64_t)(first / kLossUnit) * c.rows + row;
        if (TWO) reinterpret_cast<float4*>(c.partial)[at] = make_float4(top, rest, rest2, 0.f);
        else reinterpret_cast<float2*>(c.partial)[at] = make_float2(top, rest);
    }
}

template <bool F32, bool TWO, bool LIST>
__device__ __forceinline__ void grad_tile(const LossGemm& g, const Tile& w, const Lane& l, Control* s, uint64_t* taken) {
    const LossCall& c = g.c;
    const int row = w.m + l.row, first = g.piece0 + w.n + l.group * kLossUnit;
    const bool valid = row - g.row0[w.rank] < s->counts[w.rank];
    Listed<LIST> hit;
    hit.start(c, row, LIST && valid ? g.row0[w.rank] + c.row_token[row] : 0, first, valid && first < c.vocab);
    const float4 coef = valid ? c.coef[row] : make_float4(0.f, 0.f, 0.f, 0.f);
    const float k1 = c.k1, k2 = c.k2;
#pragma unroll 1
    for (int j = 0; j < kLossUnit / 64; ++j) {
        float v[64];
        tmem_load(v, l.tmem + j * 64);
        tmem_load(v + 32, l.tmem + j * 64 + 32);
        tmem_wait();
        if (j == kLossUnit / 64 - 1) {
            fence_before();
            warp_arrive(taken, l.lane);
        }
        const int col = first + j * 64;
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
            const Pair d = Pair(v[i], v[i + 1]) + Pair(-coef.x, -coef.x);
            Pair p = Pair(coef.y, coef.y) * exp2_of(d * Pair(k1, k1));
            if (TWO) p = p + Pair(coef.w, coef.w) * exp2_of(d * Pair(k2, k2));
            v[i] = valid && col + i < c.vocab ? p.get().x : 0.f;
            v[i + 1] = valid && col + i + 1 < c.vocab ? p.get().y : 0.f;
        }
        const Listed<LIST> before = hit;
#pragma unroll
        for (int q = 0; q < (F32 ? 3 : 1); ++q) {
            if (l.leader) tma_read_done();
            group_sync(l.group);           // the staging buffer is free
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float& lo = v[8 * i + 2 * e];
                    float& hi = v[8 * i + 2 * e + 1];
                    x[e] = bf16x2_rn(lo, hi);
                    if (F32) {
                        lo -= bf16_lo(x[e]);
                        hi -= bf16_hi(x[e]);
                    }
                }
                *reinterpret_cast<uint4*>(l.mine + ((i ^ l.turn) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
            }
            hit = before;
            while (hit.column < col + 64) {            // the exact gradient where a target or a teacher has its say
                float value = c.value[hit.at];
                for (int k = 0; k < q; ++k) value -= bf16_to_f32(f32_to_bf16_rn(value));
                const int i = hit.column - col;
                *reinterpret_cast<uint16_t*>(l.mine + (((i >> 3) ^ l.turn) << 4) + (i & 7) * 2) = f32_to_bf16_rn(value);
                hit.next();
            }
            to_async_proxy();
            group_sync(l.group);
            if (l.leader) {
                const int x = w.n + l.group * kLossUnit + j * 64, y = w.m - g.row0[0];
                tma_store_2d(&g.piece_out, l.staging, x, q * (g.row0[g.n] - g.row0[0]) + y);
                tma_commit();
            }
        }
    }
}

// What the sum over a tile's depth lost, relative to it.
__device__ __forceinline__ float cut_of(const Tile& w) { return kCutPerStep * (float)((w.k1 - w.k0) * (kTileK / 16)); }
// A gradient's factor, and what its sum lost where the tensor cores cut it (kCutPerStep) if the result is float32; of
// the six passes the last adds what counts.
template <bool F32>
__device__ __forceinline__ float factor_of(const Tile& w, const Control* s) {
    const float f = s->factors[w.rank];
    return F32 ? fmaf(f, cut_of(w), f) : f;
}

// dh: the tile goes to its split's part of acc, added there by the copy engine from the second piece on (one
// writer an element and launch, so the order is fixed).
template <bool F32>
__device__ __forceinline__ void hidden_tile(const LossGemm& g, const Tile& w, const Lane& l, uint64_t* taken) {
#pragma unroll 1
    for (int j = 0; j < kTileN / 2 / 32; ++j) {
        const int col = w.n + l.group * (kTileN / 2) + j * 32;
        float v[32];
        tmem_load(v, l.tmem + j * 32);
        tmem_wait();
        if (j == kTileN / 2 / 32 - 1) {
            fence_before();
            warp_arrive(taken, l.lane);
        }
        // the same for the whole group: no column of acc, or no depth in a shorter last piece
        if (col >= g.c.dimp || w.k1 <= w.k0) continue;
        if (l.leader) {
            if (w.more()) tma_all_done();  // the part before has been added
            else tma_read_done();
        }
        group_sync(l.group);
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = fmaf(v[i], cut_of(w), v[i]);
        }
        stage_floats(l, v);
        to_async_proxy();
        group_sync(l.group);
        if (l.leader) {
            const int y = (int)(w.split * g.c.rows) + w.m;
            if (g.add || w.more()) tma_add_2d(&g.acc, l.staging, col, y);
            else tma_store_2d(&g.acc, l.staging, col, y);
            tma_commit();
        }
    }
}

// dw: rows of the weights' gradients, rounded once.  Where rows start on 16-byte boundaries the copy engine writes
// them; else, and to add to what is there, a warp goes row by row, a lane a column.
template <bool F32>
__device__ __forceinline__ void weights_tile(const LossGemm& g, const Tile& w, const Lane& l, const Control* s, uint64_t* taken) {
    const LossCall& c = g.c;
    const float f = factor_of<F32>(w, s);
    const bool none = w.k1 <= w.k0;                    // a rank without learned tokens
    constexpr int kColumns = F32 ? 32 : 64;            // of 128 bytes
    if (g.store) {
#pragma unroll 1
        for (int j = 0; j < kTileN / 2 / kColumns; ++j) {
            float v[kColumns];
#pragma unroll
            for (int h = 0; h < kColumns / 32; ++h) tmem_load(v + h * 32, l.tmem + j * kColumns + h * 32);
            tmem_wait();
            if (j == kTileN / 2 / kColumns - 1) {
                fence_before();
                warp_arrive(taken, l.lane);
            }
            const int col = w.n + l.group * (kTileN / 2) + j * kColumns;
            if (col >= c.dim) continue;                // the same for the whole group
#pragma unroll
            for (int i = 0; i < kColumns; ++i) v[i] = none ? 0.f : f * v[i];
            if (l.leader) {
                if (F32 && w.more()) tma_all_done();
                else tma_read_done();
            }
            group_sync(l.group);
            if constexpr (F32) {
                stage_floats(l, v);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint4*>(l.mine + ((i ^ l.turn) << 4)) =
                        make_uint4(bf16x2_rn(v[8 * i], v[8 * i + 1]), bf16x2_rn(v[8 * i + 2], v[8 * i + 3]),
                                   bf16x2_rn(v[8 * i + 4], v[8 * i + 5]), bf16x2_rn(v[8 * i + 6], v[8 * i + 7]));
            }
            to_async_proxy();
            group_sync(l.group);
            if (l.leader) {
                if (F32 && w.more()) tma_add_2d(&g.out[w.rank], l.staging, col, g.piece0 + w.m);
                else tma_store_2d(&g.out[w.rank], l.staging, col, g.piece0 + w.m);
                tma_commit();
            }
        }
        return;
    }
    const int v0 = g.piece0 + w.m + l.quarter * 32;
    const int rows = min(32, min(g.piece0 + g.width, c.vocab) - v0);
    if (l.leader) tma_read_done();
    group_sync(l.group);
#pragma unroll 1
    for (int j = 0; j < kTileN / 2 / 32; ++j) {
        float v[32];
        tmem_load(v, l.tmem + j * 32);
        tmem_wait();
        if (j == kTileN / 2 / 32 - 1) {
            fence_before();
            warp_arrive(taken, l.lane);
        }
        const int col = w.n + l.group * (kTileN / 2) + j * 32;
        if (col >= c.dim) continue;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = none ? 0.f : f * v[i];
        __syncwarp();
        stage_floats(l, v);
        __syncwarp();
        const int x = col + l.lane;
        if (x >= c.dim) continue;
        constexpr int kRows = 8;                       // rows' loads at a time
        for (int i0 = 0; i0 < rows; i0 += kRows) {
            float x32[kRows];
            const int64_t at = (int64_t)(v0 + i0) * c.dim + x;
            float* out32 = static_cast<float*>(g.grads[w.rank]) + at;
            uint16_t* out16 = static_cast<uint16_t*>(g.grads[w.rank]) + at;
#pragma unroll
            for (int i = 0; i < kRows; ++i)
                x32[i] = *reinterpret_cast<const float*>(l.staging + (l.quarter * 32 + i0 + i) * 128 +
                                                       (((l.lane >> 2) ^ ((i0 + i) & 7)) << 4) + (l.lane & 3) * 4);
            if (g.accumulate || (F32 && w.more())) {
#pragma unroll
                for (int i = 0; i < kRows; ++i)
                    if (i0 + i < rows) x32[i] += F32 ? out32[(int64_t)i * c.dim] : bf16_to_f32(out16[(int64_t)i * c.dim]);
            }
#pragma unroll
            for (int i = 0; i < kRows; ++i)
                if (i0 + i < rows) {
                    if (F32) out32[(int64_t)i * c.dim] = x32[i];
                    else out16[(int64_t)i * c.dim] = f32_to_bf16_rn(x32[i]);
                }
        }
    }
}

template <LossPhase PHASE, bool F32, bool TWO, bool LIST>
__global__ void __launch_bounds__(kGemmThreads, 1) k_loss_gemm(const __grid_constant__ LossGemm g) {
    extern __shared__ char raw[];
    char* smem = raw + (1024 - (smem_of(raw) & 1023)) % 1024;
    char* staging = smem + kStages * kBytesStage;
    Control* s = reinterpret_cast<Control*>(staging + 2 * kBytesStaging);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    pdl_release();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            bar_init(&s->full[i], 1);
            bar_init(&s->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&s->ready[i], 1);
            bar_init(&s->taken[i], kEpilogueWarps);
        }
        for (int i = 0; i < kQueue; ++i) {
            bar_init(&s->tile_full[i], 1);
            bar_init(&s->tile_empty[i], kQueueReaders);
        }
        bar_init(&s->drain, 1);
        s->stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_of(&s->tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_acquire();
    if (threadIdx.x < g.n) {
        s->counts[threadIdx.x] = g.c.counts[g.first + threadIdx.x];
        if (PHASE == LossPhase::kProducts) s->factors[threadIdx.x] = g.c.factor[g.first + threadIdx.x];
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *(volatile uint32_t*)&s->tmem;
    if (warp == 0) {
        if (lane == 0) produce<PHASE, F32>(g, s, smem);
    } else if (warp == 1) {
        if (lane == 0) multiply<PHASE, F32>(g, s, smem, tmem);
    } else if (warp == 3) {
        if (lane == 0) schedule<PHASE, F32>(g, s);
    } else if (warp >= kFirstEpilogueWarp) {
        Lane l;
        l.group = (warp - kFirstEpilogueWarp) / 4;
        l.quarter = warp % 4;
        l.lane = lane;
        l.row = l.quarter * 32 + lane;
        l.staging = staging + l.group * kBytesStaging;
        l.mine = l.staging + l.row * 128;
        l.turn = l.row & 7;
        l.leader = l.row == 0;
        int buf = 0;
        uint32_t phase = 0;
        Queue queue;
        Tile w;
        while (true) {
            // one thread decides for its group, whose threads meet at barriers within a tile
            volatile int32_t* go = &s->go[l.group][buf];
            if (l.leader) {
                int state = queue.wait(s, g);
                if (state && *(volatile int32_t*)&s->queue[queue.slot].rank >= 0) state = bar_wait(&s->ready[buf], phase, s, g);
                *go = state;
            }
            group_sync(l.group);
            if (!*go) break;
            queue.read(s, &w);
            __syncwarp();
            if (lane == 0) bar_arrive(&s->tile_empty[queue.slot]);
            queue.step();
            if (w.rank < 0) break;
            fence_after();
            l.tmem = tmem + ((uint32_t)(l.quarter * 32) << 16) + buf * kTileN + l.group * (kTileN / 2);
            uint64_t* taken = &s->taken[buf];
            if (PHASE == LossPhase::kStats || PHASE == LossPhase::kKeep)
                stats_tile<F32, TWO, LIST, PHASE == LossPhase::kKeep>(g, w, l, s, taken);
            else if (PHASE == LossPhase::kGrad) grad_tile<F32, TWO, LIST>(g, w, l, s, taken);
            else if (!w.weights()) hidden_tile<F32>(g, w, l, taken);
            else weights_tile<F32>(g, w, l, s, taken);
            if (buf == 1) phase ^= 1;
            buf ^= 1;
        }
        if (l.leader) tma_all_done();
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (warp == 2) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

int64_t tile_count(LossPhase phase, const LossGemm& g) {
    int64_t rows = 0, weights = 0;
    for (int i = 0; i < g.n; ++i) rows += (g.row0[i + 1] - g.row0[i]) / kTileM;
    const int64_t columns = phase == LossPhase::kProducts ? g.c.dim : phase == LossPhase::kGrad ? g.width : g.c.vocab;
    const int64_t nt = (columns + kTileN - 1) / kTileN;
    if (phase == LossPhase::kProducts) {
        rows *= g.splits;
        weights = (int64_t)g.n * ((g.width + kTileM - 1) / kTileM);
    }
    return (rows + weights) * nt;
}

template <LossPhase PHASE, bool F32, bool TWO, bool LIST>
cudaError_t launch(const LossGemm& g, cudaStream_t stream) {
    const auto kernel = k_loss_gemm<PHASE, F32, TWO, LIST>;
    const cudaError_t e = allow_shared_memory((const void*)kernel, kSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(cap_ctas(std::min<int64_t>(tile_count(PHASE, g), sm_count()))), dim3(kGemmThreads), kSmem,
                            stream, g);
}

template <LossPhase PHASE, bool F32>
cudaError_t launch_kind(const LossGemm& g, cudaStream_t stream) {
    if (PHASE == LossPhase::kProducts) return launch<PHASE, F32, false, false>(g, stream);
    if (g.c.alpha == 0.f) return launch<PHASE, F32, false, false>(g, stream);
    if (g.c.two) return launch<PHASE, F32, true, true>(g, stream);
    return launch<PHASE, F32, false, true>(g, stream);
}

template <LossPhase PHASE>
cudaError_t launch_type(const LossGemm& g, cudaStream_t stream) {
    if (g.c.dtype == DDP_F32) return launch_kind<PHASE, true>(g, stream);
    return launch_kind<PHASE, false>(g, stream);
}

}  // namespace

cudaError_t allow_shared_memory(const void* kernel, int bytes) {
    static std::mutex lock;
    static std::set<std::pair<int, const void*>> done;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const std::lock_guard<std::mutex> hold(lock);
    if (done.count({device, kernel})) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.insert({device, kernel});
    return e;
}

cudaError_t launch_loss_gemm(LossPhase phase, const LossGemm& g, cudaStream_t stream) {
    if (tile_count(phase, g) == 0) return cudaSuccess;
    if (phase == LossPhase::kStats) return launch_type<LossPhase::kStats>(g, stream);
    if (phase == LossPhase::kKeep) return launch_type<LossPhase::kKeep>(g, stream);
    if (phase == LossPhase::kGrad) return launch_type<LossPhase::kGrad>(g, stream);
    return launch_type<LossPhase::kProducts>(g, stream);
}

}  // namespace ddpk
