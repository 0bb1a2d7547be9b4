// Attention of packed chunks of new rows over the 4-bit page cache, on the
// 5th-generation tensor cores (include/kvs.h, kvs_q4_attend_chunk).
//
// A unit of work is (sequence, kv head, query tiles): 128 rows a tile, token by
// token with the G query heads of the kv head beside each other, two tiles a
// CTA at D <= 128 and one at D = 256, against the blocks of 64 keys that some
// row of the unit sees (all up to its last row; under a window the first
// tokens' blocks, then those of the window).
//
// One CTA per SM.  All units' blocks lie in one line of cost, cut into equal
// contiguous ranges, one per CTA, whatever the sequences' lengths: a long
// history with few rows is split along its keys, short chunks share a CTA.
// Where a cut falls inside a unit its pieces leave partials (O, reference
// exponent, sum), at most two per CTA, which a second kernel joins in order.
//
// Roles:
//   softmax warps, one thread a row: load the unit's queries, then turn each
//     block's scores S in tensor memory into weights P over them, a warpgroup a
//     tile, or where there is one tile (D = 256, or few rows) both in turns, a
//     block each: a block then waits for the one before only to learn whether
//     the reference changed, which is rare; a row's
//     reference stands until the weights' sum nears f16's end, and only then is
//     the block's maximum looked for and O rescaled;
//   dequantising warps: codes and scales straight from the pages to registers
//     a block ahead, f16 values into 128-byte-swizzled stages;
//   an issuing warp per tile: S = Q K^T two blocks ahead of O += P V.
//
// Values.  A cached value is (n - 8) * scale.  The tensor core takes K and V as
// f16 values rounded once, each tile of 32 tokens brought to a common power of
// two, so that any scale the cache holds keeps f16's precision (down to 2^-12
// of what the group's largest scale reaches, and 2^-23 of it below); the power
// of two returns in the softmax, K's on the scores and V's on the weights
// before those are rounded to f16.  Queries enter as f16 times a power of two
// per row (exact down to 2^-28 of the row's largest).  (Codes as numbers, their
// scales outside the products, as one-row attention takes them, would need the
// weights once for every 32 dims.)
//
// Bound by the tensor pipe and what feeds it: 4 D operations a (row, key), the
// cache's bytes being nothing beside them from some 100 rows on.  2048 rows over
// 65536 tokens (32 / 8 heads, D 128) take 1470 us, 1.47 PFLOP/s, 76% of what
// bf16 products measure in a burst (1565 in a long run under the power cap, 80%
// of what they hold there); ncu sees the tensor pipe active on 51% of the cycles
// (1024 rows over 16384), 59% of the issue slots taken.  A block of both tiles
// takes 0.92 us; without the softmax's arithmetic and the dequantising, MMAs,
// hand-overs and loads alone, 0.69; without the dequantising 0.85, without the
// exponentials 0.78: the chain of a softmax warp (scores out of tensor memory,
// 64 exponentials, weights back) is the longest.  D 64 runs at 0.82 PFLOP/s: its
// products are half as long (tensor pipe 29%), but a block has the same chain,
// neither of whose rates is reached (31% of the exponentials', 58% of the issue
// slots); D 256 at 0.88: room for one tile only, whose chain S, softmax, P V is
// hidden by the other warpgroup's block alone.
//
// What each choice measured (2048 rows over 65536 tokens, unless said):
//   dequantising by warps of their own instead of the softmax's, one fused
//     multiply-add a pair, registers split by role: 2372 -> 1731 us;
//   a standing reference instead of a maximum every block, and tiles of 32
//     tokens in turns of four warps: 1731 -> 1580;
//   both warpgroups on a lone tile: 37 rows over 4096 tokens 34 -> 23 us, a
//     mixed batch (12 sequences, 1 to 777 rows, up to 32768 tokens) 637 -> 539;
//   rows in and out by four lanes a row (64 bytes), the next unit's queries
//     asked for early, masks only where a block needs them: the batch
//     539 -> 368, chunks of up to 1024 rows under a window of 4096 213 -> 139.
//   a worker's place in the line found by one of its warps for all: the 37 rows
//     24.2 -> 23.4, the batch 368 -> 361.  (Its first piece as well: 23.1, but
//     the batch 366 to 410, as the registers fell.)
// Blocks of 64 keys: two buffers of S and P, two O of 128 columns and Q (D 64)
// fill the 512 columns of tensor memory; 128 keys would leave one buffer each.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include <string>
#include <type_traits>

#include "kvs.h"
#include "kvs_internal.h"
#include "kvs_tcgen05.cuh"

namespace kvs {
namespace {

using namespace tc;

constexpr int kMaxSeq = 4096;
constexpr int kMaxGroup = 64;
constexpr int kWorkers = 152;  // sizes the workspace; a launch has no more CTAs
constexpr int BN = 64;         // keys of a block
constexpr int kFacs = 16;      // blocks whose factors are held: more than the stages and score buffers between the roles
constexpr float kUp = 2.f;     // a weight at the reference is 2^kUp: f16 reaches 2^13 above it and 2^26 below

struct ChunkParams {
    Q4Pool pool;
    const int32_t *table, *lens, *cu;
    int table_width, n_seq, total, G, Hq, workers;
    int window, sinks;  // window 0: none
    const void *q;
    int64_t q_stride;
    int bf16;
    float scale_log2;
    void *out;
    int64_t out_stride;
    float *lse;
    float *part_o;    // [2 * worker + (0: its first unit, begun by another; 1: its last, not ended)][tile][D / 4][row][4]
    float2 *part_ml;  // [the same][tile][row]: reference exponent and sum
    struct ChunkMeta *meta;
    int give_up;  // test hook: the MMA warps give up at their first wait, and *abort is up
    int late;     // test hook: a unit's O is read late by the warpgroup that the next unit does not begin with
};

// What a worker left for the join.
struct ChunkMeta {
    int head;  // of the unit that another worker began: 0 nothing, 1 its end, 2 a part, 3 nothing yet, it goes on
    int tail;  // 1: it began a unit that it did not end
    int h, row0, tokens;  // of that unit: kv head, first row in q, tokens
};

// ---------------------------------------------------------------- the line of work

// A unit costs kUnitCost for its beginning and end, and its keys: 1024 keys are
// 16 blocks of 0.92 us, a unit's own steps (finding it, its queries in, its
// outputs out) 13 blocks' time.  (At 512 the mixed batch's longest CTA took 1.02 M
// clocks beside a median of 0.65 M.)
constexpr int kUnitCost = 1024;
constexpr int kMinCost = 256;  // of a worker, while that leaves some idle
static_assert(BN == 64, "blocks of keys are found by shifts");

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return x < lo ? lo : (x > hi ? hi : x); }

struct Seq {
    int begin, n, T, X;  // first row, rows, cached tokens, units of a head
    int64_t pos0, cap;   // position of the first row; most keys of a unit
    int TU, some, full;  // the first unit with keys; the first with the most
    __device__ __forceinline__ void load(const ChunkParams &p, int s, int tile_tokens, int tiles) {
        begin = clampi(p.cu[s], 0, p.total);
        n = clampi(p.cu[s + 1], begin, p.total) - begin;
        const int64_t most = (int64_t)p.table_width << p.pool.lgP;
        const int len = p.lens[s];
        T = len < 0 ? 0 : (int)(len < most ? len : most);
        TU = tile_tokens * tiles;
        X = (n + TU - 1) / TU;
        pos0 = (int64_t)T - n;
        cap = (int64_t)p.window + TU + p.sinks;
        cap = p.window && cap < (int64_t)1 << 31 ? cap : (int64_t)1 << 31;
        some = pos0 >= 0 ? 0 : (int)((uint32_t)-pos0 / (uint32_t)TU);
        full = cap <= pos0 ? 0 : (int)(((uint32_t)(cap - pos0) - 1) / (uint32_t)TU);  // (rounded up, less 1)
    }
    __device__ __forceinline__ int64_t keys(int x) const {
        const int64_t k = pos0 + (int64_t)(x + 1) * TU;
        return k < 0 ? 0 : (k < cap ? k : cap);
    }
    __device__ __forceinline__ int64_t cost(int x) const { return kUnitCost + keys(x); }
    __device__ __forceinline__ int64_t before(int x) const {  // cost of units 0 .. x - 1 of a head
        const int64_t a = some < x ? some : x, b = full < a ? a : (full < x ? full : x);
        return (int64_t)x * kUnitCost + (b - a) * pos0 + TU * ((a + 1 + b) * (b - a) / 2) + (x - b) * cap;
    }
};

// blocks lo .. hi - 1 of a unit's nblk
struct Piece {
    int kind;  // 0: nothing, 1: rows that see nothing, 2: work
    int lo, hi, nblk, first, front;  // block b is keys 64 b .. for b < front, then 64 (first + b - front) ..
    int s, h, begin, n, T, x;
    int begun;  // by another worker (o1 > 0)
    int from;   // the first row's window begins here: tokens before it, but for the first `sinks`, no row of the unit sees
};

__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {  // of numbers not below 0, short where both are
    return (a | b) >> 32 ? (int64_t)((uint64_t)a / (uint64_t)b) : (int64_t)((uint32_t)a / (uint32_t)b);
}

struct Line {
    Seq q;
    int s, h, x;
    int64_t ustart, pos, end;

    // worker w of W: the equal part of the whole line that is its own.  prefix: costs of the sequences before each.
    __device__ __forceinline__ bool seek(const ChunkParams &p, const int64_t *prefix, int w, int tile_tokens, int tiles) {
        const int64_t total = prefix[p.n_seq];
        int64_t W = (total + kMinCost - 1) / kMinCost;
        W = W < p.workers ? W : p.workers;
        if (w >= W) return false;
        const int64_t each = quotient(total, W), more = total - each * W;
        pos = w * each + (w < more ? w : more);
        end = (w + 1) * each + (w + 1 < more ? w + 1 : more);
        int lo = 0, hi = p.n_seq - 1;  // the last sequence that begins at or before pos (one with rows: the next begins after)
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= pos) lo = mid;
            else hi = mid - 1;
        }
        s = lo;
        q.load(p, s, tile_tokens, tiles);
        const int64_t in = pos - prefix[s], per = q.before(q.X);
        h = (int)quotient(in, per);
        const int64_t rem = in - h * per;
        lo = 0, hi = q.X - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (q.before(mid) <= rem) lo = mid;
            else hi = mid - 1;
        }
        x = lo;
        ustart = pos - rem + q.before(x);
        return true;
    }
    __device__ __forceinline__ bool next(const ChunkParams &p, int tile_tokens, int tiles, Piece *o) {
        if (pos >= end) return false;
        const int64_t c = q.cost(x), o1 = pos - ustart, o2 = c < end - ustart ? c : end - ustart;
        const int r0 = x * q.TU, r1 = r0 + q.TU < q.n ? r0 + q.TU : q.n;
        const int64_t last = q.pos0 + r1 - 1;
        int nblk = 0, first = 0, front = 0, from = 0;
        if (last >= 0) {
            const int64_t p0 = q.pos0 + r0 < 0 ? 0 : q.pos0 + r0;
            if (p.window && p0 >= p.window) {
                from = (int)(p0 - p.window + 1);
                first = from >> 6;
                front = (p.sinks + BN - 1) >> 6;
                front = front < first ? front : first;
            }
            nblk = front + (int)(last >> 6) + 1 - first;
        }
        auto block = [&](int64_t at) {
            return at <= kUnitCost ? 0 : at == c ? nblk : (int)quotient((at - kUnitCost) * nblk, c - kUnitCost);
        };
        o->lo = block(o1);
        o->hi = block(o2);
        o->nblk = nblk;
        o->first = first;
        o->front = front;
        o->kind = o->hi > o->lo ? 2 : (nblk == 0 && o1 == 0 ? 1 : 0);
        o->begun = o1 > 0;
        o->from = from;
        o->s = s;
        o->h = h;
        o->x = x;
        o->begin = q.begin;
        o->n = q.n;
        o->T = q.T;
        pos = ustart + o2;
        if (o2 == c) {
            ustart += c;
            if (++x == q.X) {
                x = 0;
                if (++h == p.pool.Hk) {
                    h = 0;
                    while (++s < p.n_seq) {
                        q.load(p, s, tile_tokens, tiles);
                        if (q.X > 0) break;
                    }
                }
            }
        }
        return true;
    }
};

struct Walk {
    Line line;
    Piece piece;
};

// prefix[s] = cost of the sequences before s; every thread calls it
template <int kThreads>
__device__ void line_prefix(const ChunkParams &p, int tile_tokens, int tiles, int64_t *prefix) {
    __shared__ int64_t warp_sum[kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.n_seq + kThreads - 1) / kThreads;
    auto cost = [&](int s) {
        Seq q;
        q.load(p, s, tile_tokens, tiles);
        return q.before(q.X) * p.pool.Hk;
    };
    int64_t sum = 0, one = 0;
    for (int k = 0; k < per; ++k)
        if (tid * per + k < p.n_seq) sum += one = cost(tid * per + k);
    int64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int64_t base = inc - sum;
    for (int w = 0; w < warp; ++w) base += warp_sum[w];
    for (int k = 0; k < per; ++k) {
        const int s = tid * per + k;
        if (s < p.n_seq) {
            prefix[s] = base;
            base += per == 1 ? one : cost(s);
        }
    }
    if (tid == kThreads - 1) prefix[p.n_seq] = base;
    __syncthreads();
}

// ---------------------------------------------------------------- values

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t nibbles(uint32_t w) { return w & 0x00f000f0u; }

template <bool TRANS>
__device__ __forceinline__ void store_matrices(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    if (TRANS)
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                     "r"(d)
                     : "memory");
    else
        asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                     : "memory");
}
// A word of codes in each lane, its elements' scales t (times a power of two, 4 at most) in s2: four 8 x 8 matrices of
// (n - 8) t 2^-7.  A nibble ANDed out at bits 4 .. 7 and read as f16 is the subnormal n 2^-20, exactly; one fused multiply-add
// makes the value of it, rounded once: n 2^-20 * (t 2^13) - t 2^-4.  (Values below 2^-12 of the largest a group may hold are
// subnormal: off by 2^-23 of it.)
template <bool TRANS>
__device__ __forceinline__ void store_word(uint32_t addr, uint32_t w, uint32_t s2) {
    const uint32_t up = hmul2(s2, 0x70007000u), off = hmul2(s2, 0xac00ac00u);  // 2^13, -2^-4
    store_matrices<TRANS>(addr, hfma2(nibbles(w << 4), up, off), hfma2(nibbles(w >> 4), up, off), hfma2(nibbles(w), up, off),
                          hfma2(nibbles(w >> 8), up, off));
}

// ---------------------------------------------------------------- the kernel

template <int D>
struct ChunkShape {
    static constexpr int NQ = D <= 128 ? 2 : 1;         // query tiles of a CTA
    static constexpr bool kQInTmem = D != 128;          // the queries as the tensor-memory A operand, where there is room
    static constexpr int NB = D / 32;
    // warpgroups: two of softmax, two that dequantise, one whose first warps issue the MMAs
    static constexpr int kThreads = 640, kFirstDeq = 8, kFirstMma = 16;
    // of the registers at launch the softmax takes what the others leave
    static constexpr int kSoftmaxRegs = D == 256 ? 120 : 144, kDeqRegs = D == 256 ? 96 : 72, kMmaRegs = 48;
    static constexpr int kLaunchRegs = 96;
    static_assert(2 * kSoftmaxRegs + 2 * kDeqRegs + kMmaRegs <= kThreads / 128 * kLaunchRegs, "more registers than at launch are never had");
    // (giving back to a number above the launch's, or taking up to one below it, is an illegal instruction)
    static_assert(kSoftmaxRegs >= kLaunchRegs && kDeqRegs <= kLaunchRegs && kMmaRegs <= kLaunchRegs, "the softmax takes, the others give");
    static constexpr int kLines = D / 32;               // 16-byte words of codes of a lane: of a tile's K or V
    static constexpr int kStage = BN * D * 2;
    static constexpr int kStages = D == 256 ? 6 : 8;
    static constexpr int kQBytes = kQInTmem ? 0 : kTileRows * D * 2;
    static constexpr int kOffRing = NQ * kQBytes;
    static constexpr int kOffFac = kOffRing + kStages * kStage;  // K factors, V exponents, V factors [kFacs][2]
    static constexpr int kOffPiece = kOffFac + 3 * kFacs * 8;
    static constexpr int kOffBar = kOffPiece + (kThreads / 32) * (int)sizeof(Walk);
    static constexpr int kOffRows = (kOffBar + 320 + 15) / 16 * 16;  // by row: largest query element, sum [2], reference
    static constexpr int kOffStage = kOffRows + 5 * kTileRows * 4;  // 2 KB a softmax warp: 32 rows x 64 bytes on their way between memory and threads
    static constexpr int kSmem = kOffStage + 8 * 2048 + 1024;
    static_assert(kSmem <= 232448, "shared memory of a CTA");
    static constexpr uint32_t kColO = 256, kColQ = D == 256 ? 128 : 384;
    static_assert(kStages > 5, "see where the dequantising warps take turns");
    static_assert(kStages * kStage >= (kMaxSeq + 1) * 8, "the line's prefix sums lie in the ring");
};

template <int D>
__global__ void __launch_bounds__(ChunkShape<D>::kThreads, 1) chunk_kernel(const __grid_constant__ ChunkParams p) {
    using S = ChunkShape<D>;
    constexpr int NQ = S::NQ, NST = S::kStages, NB = S::NB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t bars = smem_u32(smem + S::kOffBar);
    // barriers: ring full / empty; per tile: queries there; per tile and score buffer: S full, P full, O done; the end
    auto b_full = [&](int s) { return bars + 8u * s; };
    auto b_empty = [&](int s) { return bars + 8u * (8 + s); };
    auto b_q = [&](int i) { return bars + 8u * (16 + i); };
    auto b_s = [&](int i, int buf) { return bars + 8u * (18 + 2 * i + buf); };
    auto b_p = [&](int i, int buf) { return bars + 8u * (22 + 2 * i + buf); };
    auto b_o = [&](int i, int buf) { return bars + 8u * (26 + 2 * i + buf); };
    const uint32_t b_final = bars + 8u * 30;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::kOffBar + 8 * 32);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + S::kOffBar + 8 * 33);
    float *fac_k = reinterpret_cast<float *>(smem + S::kOffFac), *exp_v = fac_k + 2 * kFacs, *fac_v = exp_v + 2 * kFacs;

    const int G = p.G, TQ = kTileRows / G, TU = NQ * TQ;
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid == 32) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(b_full(s), 2);
            mbar_init(b_empty(s), NQ);
        }
        for (int i = 0; i < 2; ++i) mbar_init(b_q(i), 8);
        for (int i = 0; i < 4; ++i) {
            mbar_init(b_s(0, i), 1);
            mbar_init(b_p(0, i), 4);
            mbar_init(b_o(0, i), 1);
        }
        mbar_init(b_final, NQ);
        *abort = p.give_up;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    int64_t *prefix = reinterpret_cast<int64_t *>(smem + S::kOffRing);
    line_prefix<S::kThreads>(p, TQ, NQ, prefix);
    // every warp walks the line by itself, its state in shared memory: lane 0 steps, the others read the piece.  (Where it
    // begins is found by one for all: by twenty at once it takes the issue slots' time.)
    Walk *walk = reinterpret_cast<Walk *>(smem + S::kOffPiece) + warp;
    if (warp == S::kFirstMma) {
        Line line;
        if (!line.seek(p, prefix, blockIdx.x, TQ, NQ)) line.pos = line.end = 0;
        if (lane < S::kThreads / 32) walk[lane - warp].line = line;
    }
    tc_before();
    __syncthreads();  // the prefix sums are read, the ring may be written
    tc_after();
    const uint32_t tmem = *tmem_slot;
    const bool any = walk->line.pos < walk->line.end;
    const Piece *piece = &walk->piece;
    auto next_piece = [&] {
        bool more = false;
        __syncwarp();
        if (any && lane == 0) {
            Line line = walk->line;  // (in registers: its fields come in together)
            Piece next;
            more = line.next(p, TQ, NQ, &next);
            if (more) walk->piece = next;
            walk->line = line;
        }
        more = __shfl_sync(0xffffffffu, more, 0);
        __syncwarp();
        return more;
    };
    // the ring's blocks in the order the MMAs take them, of a piece of n blocks: K_0, K_1, V_0, K_2, V_1, ..., V_{n-1}
    auto ring_k = [](int j) { return j < 2 ? j : 2 * j - 1; };
    auto ring_v = [](int j, int n) { return j == n - 1 ? 2 * n - 1 : 2 * j + 2; };

    if (warp >= S::kFirstMma) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kMmaRegs));
        if (warp < S::kFirstMma + NQ) {
        // ------------------------------------------------------------ MMA issue (the warp in step, one elected lane issues)
        const int i = warp - S::kFirstMma;
        constexpr uint32_t id_s = idesc(false, kTileRows, BN, false), id_o = idesc(false, kTileRows, D, true);
        const bool one = elect_one();
        const uint64_t dq = smem_desc(smem_u32(smem), 16), dk = smem_desc(smem_u32(smem + S::kOffRing), 16);
        const uint64_t dv = smem_desc(smem_u32(smem + S::kOffRing), BN * 128);
        const uint32_t tq = tmem + S::kColQ + (uint32_t)(i * D / 2);
        uint32_t ring = 0, blocks = 0, loads = 0;  // so far: stages of both tiles; blocks, query tiles of this one
        auto issue_s = [&](uint32_t r, uint32_t g) {
            const uint32_t d = tmem + (uint32_t)((2 * i + (g & 1)) * BN);
            const uint64_t db0 = dk + (uint64_t)(r % NST * S::kStage >> 4), da = dq + (uint64_t)(i * S::kQBytes >> 4);
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                const uint64_t db = db0 + (uint64_t)(((s >> 2) * (BN * 128) + (s & 3) * 32) >> 4);
                if constexpr (S::kQInTmem) mma_ts(d, tq + 8 * s, db, id_s, s > 0);
                else mma_ss(d, da + (uint64_t)(((s >> 2) * (kTileRows * 128) + (s & 3) * 32) >> 4), db, id_s, s > 0);
            }
            mma_commit(b_empty(r % NST));
            mma_commit(b_s(i, g & 1));
        };
        auto issue_o = [&](uint32_t r, uint32_t g, bool from_zero) {
            const uint32_t d = tmem + S::kColO + (uint32_t)(i * D), a = tmem + (uint32_t)((2 * i + (g & 1)) * BN);
            const uint64_t db = dv + (uint64_t)(r % NST * S::kStage >> 4);
#pragma unroll
            for (int s = 0; s < BN / 16; ++s) mma_ts(d, a + 8u * s, db + (uint64_t)(s * 2048 >> 4), id_o, !from_zero || s > 0);
            mma_commit(b_empty(r % NST));
            mma_commit(b_o(i, g & 1));
        };
        auto loaded = [&](uint32_t r) { return mbar_done(b_full(r % NST), (r / NST) & 1); };
        bool ok = !p.give_up;
        while (ok && next_piece()) {
            if (piece->kind != 2) continue;
            const int n = piece->hi - piece->lo;
            const bool active = piece->x * TU + i * TQ < piece->n;  // (else its stages are freed as they come)
            for (int j = 0; j < 2 && j < n && ok; ++j) {
                ok = wait_warp(abort, [&] { return (!active || mbar_done(b_q(i), loads & 1)) & loaded(ring + ring_k(j)); });
                if (!ok) break;
                tc_after();
                if (one) {
                    if (active) issue_s(ring + ring_k(j), blocks + j);
                    else mma_commit(b_empty((ring + ring_k(j)) % NST));
                }
            }
            // S_{j+2} takes the buffer of S_j and P_j: P_j was read by O's MMA before it, and the pipe keeps their order
            for (int j = 0; j < n && ok; ++j) {
                const bool more = j + 2 < n;
                const uint32_t rv = ring + ring_v(j, n), rk = ring + ring_k(j + 2);
                ok = wait_warp(abort, [&] {
                    bool all = loaded(rv);
                    if (active) all &= mbar_done(b_p(i, (blocks + j) & 1), ((blocks + j) >> 1) & 1);
                    if (more) all &= loaded(rk);
                    return all;
                });
                if (!ok) break;
                tc_after();
                if (one) {
                    if (active) {
                        issue_o(rv, blocks + j, j == 0);
                        if (more) issue_s(rk, blocks + j + 2);
                    } else {
                        mma_commit(b_empty(rv % NST));
                        if (more) mma_commit(b_empty(rk % NST));
                    }
                }
            }
            ring += 2 * n;
            if (active) blocks += n, ++loads;
        }
        if (one) mma_commit(b_final);  // on every path: tensor memory is freed only after it
        }
    } else if (warp >= S::kFirstDeq) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kDeqRegs));
        // ------------------------------------------------------------ pages to f16 stages: half of the warps K, half V
        // a tile of 32 tokens at a time, every other block's first or second
        constexpr int kPer = NB / 2;  // pairs of 32-dim blocks
        const int dw = warp - S::kFirstDeq, side = dw & 1, turn = dw >> 1 & 1;
        const bool is_v = dw >= 4;
        const int g = lane >> 2, t = lane & 3, m = lane >> 3, r8 = lane & 7;
        const int lg = p.pool.lgP - 5, D36 = 36 * D;
        const uint32_t ring_base = smem_u32(smem + S::kOffRing) + (uint32_t)(side * 32 * 128);
        uint32_t ring = 0, blocks = 0;
        bool ok = true;
        while (ok && next_piece()) {
            if (piece->kind != 2) continue;
            const int lo = piece->lo, n = piece->hi - lo, front = piece->front, first = piece->first, T = piece->T, h = piece->h;
            const int from = piece->from;
            const int32_t *table = p.table + (int64_t)piece->s * p.table_width;
            int page_base = -32, page = -1;
            // block j's tile: its bytes, tokens from its first on (0 and less: none that counts), and whether its page lies
            // outside the pool.  Bytes are always some of the pool's, so that the loads need no branch: values merged from
            // two sides are copied, and a copy waits for its load.
            struct Where {
                const uint8_t *at;
                int left;
                bool bad;
            };
            auto where = [&](int j) {
                const int b = lo + j, kt = 2 * (b < front ? b : first + b - front) + side;
                Where w;
                w.left = T - kt * 32;
                if ((kt + 1) * 32 <= from && kt * 32 >= p.sinks) w.left = 0;  // no row sees it: its page may be gone
                w.at = p.pool.pages;
                w.bad = false;
                if (w.left > 0) {
                    const int pg = kt >> lg;
                    if (pg < page_base || pg >= page_base + 32) {
                        page_base = pg;
                        page = pg + lane < p.table_width ? table[pg + lane] : -1;
                    }
                    const int num = __shfl_sync(0xffffffffu, page, pg - page_base);
                    w.bad = num < 0 || num >= p.pool.n_pages;
                    if (!w.bad) w.at += num * p.pool.page_bytes + h * p.pool.head_bytes + (kt & ((1 << lg) - 1)) * D36;
                }
                return w;
            };
            uint4 code[S::kLines];
            auto line = [&](const uint8_t *at, int i) { return __ldg(reinterpret_cast<const uint4 *>(at) + i * 32 + lane); };
            // the tile's largest scale is below 2^(E + 1): factor 2^(1 - E) as two f16
            auto common = [&](__half2 most, int &E) {
                uint32_t x = *reinterpret_cast<uint32_t *>(&most);
                x = (x & 0xffffu) > (x >> 16) ? (x & 0xffffu) : (x >> 16);
                x = __reduce_max_sync(0xffffffffu, x);
                const int field = (int)(x >> 10) > 1 ? (int)(x >> 10) : 1;  // (31: an infinity)
                E = field - 15;
                const uint32_t f = field >= 31 ? 0x0200u : (uint32_t)(31 - field) << 10;
                return f | f << 16;
            };
            auto larger = [](__half2 a, uint32_t w) { return __hmax2(a, __habs2(*reinterpret_cast<const __half2 *>(&w))); };
            auto wait_free = [&](uint32_t r) {
                if (r >= (uint32_t)NST) ok = mbar_wait_warp(b_empty(r % NST), (r / NST - 1) & 1, abort);
                return ok;
            };
            auto publish = [&](uint32_t r) {
                proxy_fence();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_full(r % NST));
            };
            auto word = [](const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; };
            // Every other block of the CTA is this warp's, whichever unit it is of: a warp's items are then at most 5 places of
            // the ring apart, and a stage that it waits for has no phase behind the last but one that it has not seen complete.
            const int j0 = (turn ^ (int)blocks) & 1;
            if (j0 >= n) {
                ring += 2 * n;
                blocks += n;
                continue;
            }
            // the next tile's bytes are fetched as soon as a tile's are converted (past the last, some again)
            Where cur = where(j0), next = j0 + 2 < n ? where(j0 + 2) : cur;
            if (!is_v) {
                // a lane's words: of tokens 8 x + g; scales of tokens 16 c + g and 16 c + 8 + g in a word
                // (kept as loaded, and copied before they are changed: a value changed in place is moved at the loop's end, and
                // the move waits for its load)
                using Scales = std::conditional_t<D == 64, uint2, uint4>;
                constexpr int kVecs = NB * 4 / (int)sizeof(Scales);
                Scales held[2][kVecs];
                auto fetch = [&](const uint8_t *at) {
#pragma unroll
                    for (int x = 0; x < S::kLines; ++x) code[x] = line(at, x);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int x = 0; x < kVecs; ++x) held[c][x] = __ldg(reinterpret_cast<const Scales *>(at + 16 * D + (c * 8 + g) * NB * 4) + x);
                };
                fetch(cur.at);
                const uint32_t at_k = (uint32_t)(r8 * 128 + ((m ^ r8) << 4));  // a lane's row of a matrix: token r8 of 8
                for (int j = j0; j < n; j += 2) {
                    const uint32_t r = ring + ring_k(j);
                    if (!wait_free(r)) break;
                    uint32_t sc[2][NB];
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int b = 0; b < NB; ++b) sc[c][b] = reinterpret_cast<const uint32_t *>(held[c])[b];
                    if (cur.left < 32 || cur.bad) {  // tokens past the last count as 0, a page outside the pool as NaN
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const uint32_t keep = (16 * c + g < cur.left ? 0xffffu : 0u) | (16 * c + g + 8 < cur.left ? 0xffff0000u : 0u);
#pragma unroll
                            for (int b = 0; b < NB; ++b) sc[c][b] = (sc[c][b] | (cur.bad ? 0x7e007e00u : 0u)) & keep;
                        }
                    }
                    __half2 most = __half2half2(__ushort_as_half(0));
#pragma unroll
                    for (int b = 0; b < 2 * NB; ++b) most = larger(most, sc[b / NB][b % NB]);
                    int E;
                    const uint32_t f2 = common(most, E), dst = ring_base + r % NST * S::kStage + at_k;
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const uint32_t s = hmul2(sc[c][b], f2);
#pragma unroll
                            for (int y = 0; y < 2; ++y) {  // 8 tokens
                                const int x = 2 * c + y;
                                const uint32_t w = D == 64 ? word(code[c], 2 * y + b) : word(code[x * (NB / 4) + b / 4], b % 4);
                                store_word<false>((dst + x * 1024 + (b >> 1) * (BN * 128)) ^ ((b & 1) << 6), w, __byte_perm(s, 0, y ? 0x3232 : 0x1010));
                            }
                        }
                    if (lane == 0) fac_k[(blocks + j) % kFacs * 2 + side] = __uint_as_float((uint32_t)(127 + E + 6) << 23);
                    publish(r);
                    cur = next;
                    fetch(cur.at);
                    if (j + 4 < n) next = where(j + 4);
                }
            } else {
                // a lane's words: dims g, g + 8, g + 16, g + 24 of a block, tokens 16 c + 4 t .. + 3 in pairs; scales of the
                // pairs (0, 1), (2, 3) of a block and of the next
                uint4 held[2][D / 64];
                auto fetch = [&](const uint8_t *at) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
#pragma unroll
                        for (int x = 0; x < kPer; ++x) code[c * kPer + x] = line(at + 18 * D, c * kPer + x);
                        const uint4 *src = reinterpret_cast<const uint4 *>(at + 34 * D + (c * 4 + t) * NB * 8);
#pragma unroll
                        for (int x = 0; x < D / 64; ++x) held[c][x] = __ldg(src + x);
                    }
                };
                fetch(cur.at);
                const int vt = 4 * (r8 >> 1) + (r8 & 1);  // a lane's row of a matrix: token 4 (r8 / 2) + r8 % 2 of the 16 (+ 2)
                const uint32_t at_v[2] = {(uint32_t)(vt * 128 + ((m ^ (vt & 7)) << 4)), (uint32_t)((vt + 2) * 128 + ((m ^ ((vt + 2) & 7)) << 4))};
                for (int j = j0; j < n; j += 2) {
                    const uint32_t r = ring + ring_v(j, n);
                    if (!wait_free(r)) break;
                    uint4 sc[2][D / 64];
#pragma unroll
                    for (int x = 0; x < 2 * (D / 64); ++x) sc[x / (D / 64)][x % (D / 64)] = held[x / (D / 64)][x % (D / 64)];
                    if (cur.left < 32 || cur.bad) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int left = cur.left - 16 * c - 4 * t;
                            const uint32_t k0 = (left > 0 ? 0xffffu : 0u) | (left > 1 ? 0xffff0000u : 0u), k1 = (left > 2 ? 0xffffu : 0u) | (left > 3 ? 0xffff0000u : 0u);
                            const uint32_t wrong = cur.bad ? 0x7e007e00u : 0u;
#pragma unroll
                            for (int x = 0; x < D / 64; ++x) {
                                uint4 &v = sc[c][x];
                                v.x = (v.x | wrong) & k0, v.y = (v.y | wrong) & k1, v.z = (v.z | wrong) & k0, v.w = (v.w | wrong) & k1;
                            }
                        }
                    }
                    __half2 most = __half2half2(__ushort_as_half(0));
#pragma unroll
                    for (int x = 0; x < 2 * (D / 64); ++x) {
                        const uint4 &v = sc[x / (D / 64)][x % (D / 64)];
                        most = larger(larger(larger(larger(most, v.x), v.y), v.z), v.w);
                    }
                    int E;
                    const uint32_t f2 = common(most, E), dst = ring_base + r % NST * S::kStage;
#pragma unroll
                    for (int x = 0; x < S::kLines; ++x) {  // two 32-dim blocks of 16 tokens
                        const int c = x / kPer, pair = x % kPer;
#pragma unroll
                        for (int y = 0; y < 4; ++y)  // block y / 2 of them, token pairs y % 2
                            store_word<true>(dst + c * 2048 + pair * (BN * 128) + (at_v[y & 1] ^ ((y >> 1) << 6)), word(code[x], y), hmul2(word(sc[c][pair], y), f2));
                    }
                    if (lane == 0) {
                        exp_v[(blocks + j) % kFacs * 2 + side] = (float)(E + 6);
                        fac_v[(blocks + j) % kFacs * 2 + side] = __uint_as_float((uint32_t)(127 - 6 - E) << 23);
                    }
                    publish(r);
                    cur = next;
                    fetch(cur.at);
                    if (j + 4 < n) next = where(j + 4);
                }
            }
            ring += 2 * n;
            blocks += n;
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kSoftmaxRegs));
        // ------------------------------------------------------------ softmax, one thread per row
        const int wg = warp >> 2, row = tid & 127, hg = row % G;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const float nan = __int_as_float(0x7fc00000);
        uint32_t *tops = reinterpret_cast<uint32_t *>(smem + S::kOffRows);
        float *row_sum = reinterpret_cast<float *>(tops + 2 * kTileRows) + row, *row_ref = row_sum + 2 * kTileRows;
        auto out_of_q = [&](int64_t trow, int hq) { return static_cast<const uint16_t *>(p.q) + (trow * p.q_stride + (int64_t)hq * D); };
        float fac = 0.f;
        uint32_t ring = 0, blocks0 = 0, blocks1 = 0, all_blocks = 0;  // so far: stages, blocks of tile 0, of tile 1, of the CTA
        bool ok = true;  // (every warp goes on to the end of the line whatever it has given up: the barriers count them all)
        ChunkMeta meta = {};
        // barriers of both warpgroups: all; "block done" of warpgroup wg
        auto sync_all = [] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
        auto done_wait = [&] { asm volatile("bar.sync %0, 256;" ::"r"(3 - wg) : "memory"); };
        auto done_tell = [&] { asm volatile("bar.arrive %0, 256;" ::"r"(2 + wg) : "memory"); };
        // "O is read", across a change of unit: the next unit's first P V writes tile 0's O anew as soon as one warpgroup has
        // published its first weights, and where either unit is on one tile the other may have columns of that O to read.  So
        // the one that publishes them waits for the other's word: always in a unit on one tile (the first takes it too, from
        // nobody's reading), and in one on two tiles that follows such a unit.  (Two uses of the barrier have a sync_all between
        // them, which both pass after the first.)
        bool hear = false;  // of warpgroup 0: the unit on two tiles follows one on one
        auto read_tell = [] { asm volatile("bar.arrive 4, 256;" ::: "memory"); };
        auto read_wait = [] {
            asm volatile("bar.sync 4, 256;" ::: "memory");
            tc_after();
        };
        auto hear_read = [&] {
            if (hear) read_wait();
            hear = false;
        };
        auto one_tile = [&](const Piece &c) { return NQ == 1 || c.x * TU + TQ >= c.n; };  // both warpgroups on tile 0
        // 16 bytes k of row r of the warp's stage, where 8 neighbours read or write all banks once
        uint4 *stage = reinterpret_cast<uint4 *>(smem + S::kOffStage + warp * 2048);
        auto staged = [&](int r, int k) { return stage + r * 4 + (k ^ (r >> 1 & 3)); };
        // The unit's queries as f16 times a power of two a row, dims of each 32-dim block in the order of a K row: even ones of
        // the first 16, odd ones, even ones of the last 16, odd ones.  A warpgroup loads its tile's; with one tile half of the
        // dims each (D 64: the first all).  Four lanes read 64 bytes of a row, and a row's thread gets them through the warp's
        // stage.
        auto load_dims = [&](auto dims, const Piece &c, int tile, int d0, bool mine, bool shared) {
            constexpr int N = decltype(dims)::value;
            uint4 v[N / 8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = (row & 96) + 8 * k + (lane >> 2), tok = c.x * TU + tile * TQ + r / G;
                const bool valid = mine && r < TQ * G && tok < c.n;
                const uint4 *src = reinterpret_cast<const uint4 *>(out_of_q(valid ? c.begin + tok : 0, valid ? c.h * G + r % G : 0) + d0 + 8 * (lane & 3));
#pragma unroll
                for (int x = 0; x < N / 32; ++x) v[4 * x + k] = valid ? __ldg(src + 4 * x) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int x = 0; x < N / 32; ++x) {
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 4; ++k) *staged(8 * k + (lane >> 2), lane & 3) = v[4 * x + k];
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 4; ++k) v[4 * x + k] = *staged(lane, k);
            }
            uint32_t top2 = 0;
#pragma unroll
            for (int x = 0; x < N / 8; ++x) {
                top2 = __vmaxu2(__vmaxu2(top2, v[x].x & 0x7fff7fffu), v[x].y & 0x7fff7fffu);
                top2 = __vmaxu2(__vmaxu2(top2, v[x].z & 0x7fff7fffu), v[x].w & 0x7fff7fffu);
            }
            uint32_t top = max(top2 & 0xffffu, top2 >> 16);
            if (shared) {
                tops[wg * kTileRows + row] = top;
                sync_all();
                top = max(tops[row], tops[kTileRows + row]);
            }
            const float top_f = p.bf16 ? __uint_as_float(top << 16) : __half2float(__ushort_as_half((unsigned short)top));
            int e = (int)(__float_as_uint(top_f) >> 23) - 127;
            e = e < -100 ? -100 : (e > 100 ? 100 : e);
            const float f = copysignf(__uint_as_float((uint32_t)(127 + 14 - e) << 23), p.scale_log2);
            // never 0, so that a masked score stays -inf times it
            fac = fmaxf(fabsf(p.scale_log2) * __uint_as_float((uint32_t)(127 - 14 + e) << 23), 1.17549435e-38f);
            auto two = [&](uint32_t w) {
                const float2 y = p.bf16 ? make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u))
                                        : __half22float2(*reinterpret_cast<const __half2 *>(&w));
                return make_float2(y.x * f, y.y * f);
            };
            if (mine) {
#pragma unroll
                for (int b2 = 0; b2 < N / 64; ++b2) {
                    uint32_t o[32];
#pragma unroll
                    for (int x = 0; x < 8; ++x) {  // 8 dims: half of the even and of the odd chunk of 16
                        const uint4 u = v[8 * b2 + x];
                        const float2 a = two(u.x), b = two(u.y), c2 = two(u.z), d = two(u.w);
                        uint32_t *at = o + (x >> 1) * 8 + (x & 1) * 2;
                        at[0] = pack<false>(a.x, b.x), at[1] = pack<false>(c2.x, d.x);
                        at[4] = pack<false>(a.y, b.y), at[5] = pack<false>(c2.y, d.y);
                    }
                    const int g64 = d0 / 64 + b2;
                    if constexpr (S::kQInTmem) {
                        tmem_st32(lanes + S::kColQ + (uint32_t)(tile * D / 2 + g64 * 32), o);
                    } else {
                        uint8_t *dst = smem + tile * S::kQBytes + g64 * (kTileRows * 128) + row * 128;
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            *reinterpret_cast<uint4 *>(dst + ((x ^ (row & 7)) << 4)) = make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
                    }
                }
            }
            if constexpr (S::kQInTmem) {
                tmem_wait_st();
                tc_before();
            } else {
                proxy_fence();
            }
            __syncwarp();
            if (lane == 0) {  // 8 arrivals a tile
                mbar_arrive(b_q(tile));
                if (!shared) mbar_arrive(b_q(tile));
            }
        };
        auto load_queries = [&](const Piece &c) {
            if (one_tile(c)) {
                if constexpr (D == 64) load_dims(std::integral_constant<int, 64>{}, c, 0, 0, wg == 0, true);
                else load_dims(std::integral_constant<int, D / 2>{}, c, 0, wg * (D / 2), true, true);
            } else if constexpr (NQ == 2) {
                load_dims(std::integral_constant<int, D>{}, c, wg, 0, true, false);
            }
        };
        // the queries of the piece after this one, towards the caches: a line a lane
        auto expect_queries = [&](const Piece &c) {
            constexpr int kLinesOfRow = D / 64;  // of 128 bytes
            for (int x = tid & 255; x < NQ * kTileRows * kLinesOfRow; x += 256) {
                const int r = x / kLinesOfRow, tile = r / kTileRows, tok = c.x * TU + tile * TQ + r % kTileRows / G;
                if (r % kTileRows < TQ * G && tok < c.n)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(out_of_q(c.begin + tok, c.h * G + r % kTileRows % G) + 64 * (x % kLinesOfRow)));
            }
        };
        auto out_row = [&](int64_t trow, int hq) { return static_cast<uint16_t *>(p.out) + (trow * p.out_stride + (int64_t)hq * D); };
        // the next piece with work, rows that see nothing written on the way
        auto find_work = [&] {
            while (next_piece()) {
                const Piece &c = *piece;
                if (warp == 0) {
                    if (c.begun && c.lo > 0) meta.head = c.kind == 2 ? (c.hi == c.nblk ? 1 : 2) : (c.lo < c.nblk ? 3 : 0);
                    if (c.kind == 2 && c.lo == 0 && c.hi < c.nblk) {
                        meta.tail = 1;
                        meta.h = c.h;
                        meta.row0 = c.begin + c.x * TU;
                        meta.tokens = min(TU, c.n - c.x * TU);
                    }
                }
                if (c.kind == 2) return true;
                const int tok = c.x * TU + wg * TQ + row / G;
                if (c.kind == 1 && wg < NQ && row < TQ * G && tok < c.n) {
                    const int64_t trow = c.begin + tok;
                    const int hq = c.h * G + hg;
                    uint4 *dst = reinterpret_cast<uint4 *>(out_row(trow, hq));
                    for (int x = 0; x < D / 8; ++x) dst[x] = make_uint4(0, 0, 0, 0);
                    if (p.lse) p.lse[trow * p.Hq + hq] = -INFINITY;
                }
            }
            return false;
        };
        bool work = find_work();
        if (work) load_queries(*piece);
        if (work && one_tile(*piece) && wg == 1) read_tell();  // there is nothing to read yet
        while (work) {
            const Piece c = *piece;
            __syncwarp();
            work = find_work();  // the next
            if (work) expect_queries(*piece);
            const bool shared = one_tile(c);
            const int i = shared ? 0 : wg;  // the tile
            const int n = c.hi - c.lo, ft = c.x * TU + i * TQ, tok = ft + row / G;
            const bool valid = row < TQ * G && tok < c.n;
            const int pos0 = c.T - c.n, pos = pos0 + tok;
            const int pf = pos0 + ft, pl = max(pos0 + min(ft + TQ, c.n) - 1, -1);  // positions of the tile's first and last row
            const int masked_from = ((pf + 1) >> 6) - c.first + c.front - c.lo;  // (pf + 1) / BN: blocks from there reach past a row
            // and under a window the first tokens' blocks and those where some row's window begins
            const int masked_to = p.window ? max(((pl - p.window) >> 6) + 1 - c.first, 0) + c.front - c.lo : 0;
            const uint32_t first_block = i ? blocks1 : blocks0;
            float m = -INFINITY, l = 0.f;
            // what a block needs beside its scores: K's factors times the row's, V's exponents and their factors, of its two tiles
            struct Factors {
                float sc[2], ex[2], vf[2];
            };
            auto factors = [&](int j) {
                const int slot = (all_blocks + j) % kFacs;
                const float2 k = *reinterpret_cast<const float2 *>(fac_k + 2 * slot), x = *reinterpret_cast<const float2 *>(exp_v + 2 * slot);
                const float2 v = *reinterpret_cast<const float2 *>(fac_v + 2 * slot);
                return Factors{{fac * k.x, fac * k.y}, {x.x, x.y}, {v.x, v.y}};
            };
            auto scores_at = [&](int j) { return lanes + (uint32_t)((2 * i + ((first_block + j) & 1)) * BN); };
            auto ready = [&](int j) {
                const uint32_t gb = first_block + j, rv = ring + ring_v(j, n);
                return mbar_done(b_s(i, gb & 1), (gb >> 1) & 1) & mbar_done(b_full(rv % NST), (rv / NST) & 1);
            };
            float s[BN];
            uint32_t pk[BN / 2];
            float part[2];  // sums of the two tiles' weights
            auto load_half = [&](int j, int x) { tmem_ld32(scores_at(j) + 32 * x, reinterpret_cast<uint32_t *>(s) + 32 * x); };
            auto mask = [&](int j, int h) {  // of 32 keys
                if (j < masked_from && j >= masked_to) return;
                const int b = c.lo + j, k0 = (b < c.front ? b : c.first + b - c.front) * BN + 32 * h;
                if (j >= masked_from) {  // some row of the tile ends inside the block
                    const int lim = pos - k0;
#pragma unroll
                    for (int x = 0; x < 32; ++x) s[32 * h + x] = x <= lim ? s[32 * h + x] : -INFINITY;
                }
                if (p.window && k0 <= pl - p.window && k0 + 32 > p.sinks) {  // some row's window begins inside them or after
                    const int begin = (pos > -1 ? pos : -1) - p.window - k0, sk = p.sinks - k0;
#pragma unroll
                    for (int x = 0; x < 32; ++x) s[32 * h + x] = x > begin || x < sk ? s[32 * h + x] : -INFINITY;
                }
            };
            auto load_scores = [&](int j) {
                load_half(j, 0);
                load_half(j, 1);
                tmem_wait_ld();
                mask(j, 0);
                mask(j, 1);
            };
            auto weights = [&](const Factors &f, int x) {  // of 32 keys
                const float neg = (m == -INFINITY ? 0.f : kUp - m) + f.ex[x];
                const float2 sc2 = make_float2(f.sc[x], f.sc[x]), neg2 = make_float2(neg, neg);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int y = 0; y < 32; y += 2) {
                    const float2 z = fma2(make_float2(s[32 * x + y], s[32 * x + y + 1]), sc2, neg2);
                    const float2 e = make_float2(ex2(z.x), ex2(z.y));
                    sum[y >> 1 & 1] = add2(sum[y >> 1 & 1], e);
                    pk[16 * x + y / 2] = pack<false>(e.x, e.y);
                }
                const float2 both = add2(sum[0], sum[1]);
                part[x] = both.x + both.y;
            };
            // The weights' sum bounds each of them: while it is below 2^15 none passes f16, and the reference (a maximum seen
            // before) stands.  Else, and for a row's first key, the block's maximum (of scores loaded again) becomes it and the weights are formed anew; false: a wait
            // gave up.
            auto must_grow = [&] { return __any_sync(0xffffffffu, m == -INFINITY || !(part[0] + part[1] <= 32768.f)); };
            auto grow_reference = [&](int j, const Factors &f) {
                const bool over = m == -INFINITY || !(part[0] + part[1] <= 32768.f);
                float top[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float a[2] = {fmaxf(s[32 * x], s[32 * x + 1]), fmaxf(s[32 * x + 2], s[32 * x + 3])};
#pragma unroll
                    for (int y = 4; y < 32; y += 2) a[y >> 1 & 1] = fmax3(a[y >> 1 & 1], s[32 * x + y], s[32 * x + y + 1]);
                    top[x] = fmaf(fmaxf(a[0], a[1]), f.sc[x], f.ex[x]);
                }
                const float mx = fmaxf(top[0], top[1]);
                // (from 2^1 on, so that 64 weights at the reference are far below the bound)
                const bool grow = over && (m == -INFINITY ? mx != -INFINITY : mx > m + 1.f);
                bool done = true;
                if (__any_sync(0xffffffffu, grow)) {
                    const float to = grow ? mx : m;
                    const float alpha = m == -INFINITY ? 0.f : ex2(m - to);
                    l *= alpha;
                    m = to;
                    if (j > 0) {
                        const uint32_t before = first_block + j - 1;
                        done = mbar_wait_warp(b_o(i, before & 1), (before >> 1) & 1, abort);
                        tc_after();
                        const uint32_t to_o = lanes + S::kColO + (uint32_t)(i * D);
#pragma unroll 1
                        for (int x = 0; x < D && done; x += 16) {
                            uint32_t v[16];
                            tmem_ld16(to_o + x, v);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
                            tmem_st16(to_o + x, v);
                        }
                    }
                }
                return done;
            };
            auto publish = [&](int j, const Factors &f) {
                tmem_st32(scores_at(j), pk);
                l += part[0] * f.vf[0] + part[1] * f.vf[1];  // (without V's powers of two)
                tmem_wait_st();
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_p(i, (first_block + j) & 1));
            };
            if (shared) {
                for (int j = (first_block & 1) == (uint32_t)wg ? 0 : 1; j < n; j += 2) {
                    if (ok) ok = wait_warp(abort, [&] { return ready(j); });
                    tc_after();
                    const Factors f = factors(j);
                    bool before = j > 0, grown = false;  // the block before is yet to be heard of; the reference has grown for this one
                    do {
                        if (ok) {
                            load_scores(j);  // (S stays until its P is stored)
                            weights(f, 0);
                            weights(f, 1);
                        }
                        if (before) {  // it is done: its reference is the one that stands
                            before = false;
                            done_wait();
                            const float now = *row_ref;
                            const bool stale = now != m;
                            if (stale) {
                                l = m == -INFINITY ? l : l * ex2(m - now);
                                m = now;
                            }
                            if (__any_sync(0xffffffffu, stale)) continue;
                        }
                        if (!ok || grown || !must_grow()) break;
                        load_scores(j);
                        ok = grow_reference(j, f);
                        grown = true;
                    } while (true);
                    if (j == 0) read_wait();
                    if (ok) publish(j, f);
                    *row_ref = m;
                    if (j + 1 < n) done_tell();
                }
            } else {
                for (int j = 0; j < n && ok; ++j) {
                    ok = wait_warp(abort, [&] { return ready(j); });
                    if (!ok) break;
                    tc_after();
                    const Factors f = factors(j);
                    for (bool grown = false;; grown = true) {
                        load_scores(j);  // (S stays until its P is stored)
                        weights(f, 0);
                        weights(f, 1);
                        if (grown || !must_grow()) break;
                        load_scores(j);
                        ok = grow_reference(j, f);
                        if (!ok) break;
                    }
                    if (!ok) break;
                    hear_read();
                    publish(j, f);
                }
                hear_read();  // (a wait gave up before: the other's word is taken all the same)
            }
            ring += 2 * n;
            all_blocks += n;
            blocks0 += n;
            if (!shared) blocks1 += n;
            const uint32_t last = (i ? blocks1 : blocks0) - 1;
            if (shared) {  // both are done with the scores, the reference is the last one
                sync_all();
                const float now = *row_ref;
                // (without a reference the sum is 0, or NaN where every key that the row saw was)
                row_sum[wg * kTileRows] = !ok ? nan : m == -INFINITY ? l : l * ex2(m - now);
                m = now;
            }
            // the next queries go in before this unit's output comes out: its scores are all read
            if (work) load_queries(*piece);
            if (shared) {
                sync_all();
                l = row_sum[0] + row_sum[kTileRows];
            }
            if (ok) ok = mbar_wait_warp(b_o(i, last & 1), (last >> 1) & 1, abort);
            tc_after();
            if (!ok) l = nan;
            // the other warpgroup has tile 0's first block of the next unit: it is to know when this one has read
            const bool next_shared = work && one_tile(*piece);
            const bool tell = next_shared ? wg != (int)(blocks0 & 1) : work && shared && wg == 1;
            hear = work && shared && !next_shared && wg == 0;
            if (p.late && tell)
                for (int k = 0; k < 50; ++k) __nanosleep(1000);
            const bool whole = c.lo == 0 && c.hi == c.nblk;
            const uint32_t to = lanes + S::kColO + (uint32_t)(i * D);
            const int x0 = shared ? wg * (D / 2) : 0, x1 = shared ? x0 + D / 2 : D;
            auto was_read = [&](int x) {  // with the columns from x on
                if (!tell || x + 32 < x1) return;
                tc_before();
                read_tell();
            };
            if (whole) {
                const int64_t trow = c.begin + tok;
                const int hq = c.h * G + hg;
                const float inv = 1.f / l;
                // rows go out through the warp's stage as the queries came in, 64 bytes of a row by four lanes
                uint16_t *dst[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = (row & 96) + 8 * k + (lane >> 2), rtok = ft + r / G;
                    dst[k] = r < TQ * G && rtok < c.n ? out_row(c.begin + rtok, c.h * G + r % G) + 8 * (lane & 3) : nullptr;
                }
#pragma unroll 1
                for (int x = x0; x < x1; x += 32) {
                    uint32_t v[32] = {};
                    if (ok) {  // (the same in a warp; else MMAs may be under way, and what they have is not wanted)
                        tmem_ld32(to + x, v);
                        tmem_wait_ld();
                    }
                    was_read(x);
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        uint32_t o[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            // a row that saw nothing: out 0, lse -inf
                            const float a = l == 0.f ? 0.f : __uint_as_float(v[k + 2 * y]) * inv;
                            const float z = l == 0.f ? 0.f : __uint_as_float(v[k + 2 * y + 1]) * inv;
                            o[y] = p.bf16 ? pack<true>(a, z) : pack<false>(a, z);
                        }
                        *staged(lane, k / 8) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (dst[k]) *reinterpret_cast<uint4 *>(dst[k] + x) = *staged(8 * k + (lane >> 2), lane & 3);
                }
                if (valid && x0 == 0 && p.lse) p.lse[trow * p.Hq + hq] = l == 0.f ? -INFINITY : (m + log2f(l) - kUp) * 0.693147180559945309f;
            } else {
                const int64_t at = (int64_t)(2 * (int)blockIdx.x + (c.lo == 0)) * NQ + i;
                float4 *dst = reinterpret_cast<float4 *>(p.part_o) + at * (D / 4 * kTileRows) + row;
#pragma unroll 1
                for (int x = x0; x < x1; x += 32) {
                    uint32_t v[32] = {};
                    if (ok) {
                        tmem_ld32(to + x, v);
                        tmem_wait_ld();
                    }
                    was_read(x);
                    if (valid) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            dst[(x + k) / 4 * kTileRows] = make_float4(__uint_as_float(v[k]), __uint_as_float(v[k + 1]),
                                                                       __uint_as_float(v[k + 2]), __uint_as_float(v[k + 3]));
                    }
                }
                if (valid && x0 == 0) p.part_ml[at * kTileRows + row] = make_float2(m, l);
            }
        }
        if (tid == 0) p.meta[blockIdx.x] = meta;
    }
    // tensor memory is freed once every MMA is done and every row was read
    if (tid == 0) mbar_drain(b_final, 0);
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// Joins the partials of a unit that several workers shared, in the line's
// order.  blockIdx.x: the worker that began it, blockIdx.y: tile and 16 dims;
// one thread per row.
constexpr int kJoinDims = 16;
constexpr int kJoinAtOnce = 4;  // partials a thread has on their way
template <int D>
__global__ void __launch_bounds__(kTileRows) join_kernel(const __grid_constant__ ChunkParams p) {
    constexpr int NQ = ChunkShape<D>::NQ;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // on every path: the call ends after the attention has
    const int w = blockIdx.x, i = (int)blockIdx.y % NQ, d0 = (int)blockIdx.y / NQ * kJoinDims, row = threadIdx.x;
    const ChunkMeta meta = p.meta[w];
    const int TQ = kTileRows / p.G, tok = i * TQ + row / p.G;
    if (!meta.tail) return;
    const bool mine = row < TQ * p.G && tok < meta.tokens;
    float m = -INFINITY, l = 0.f;
    float4 o[kJoinDims / 4] = {};
    float2 ml[kJoinAtOnce];
    float4 v[kJoinAtOnce][kJoinDims / 4];
    auto fetch = [&](int k, int slot, bool there) {
        const int64_t at = (int64_t)slot * NQ + i;
        ml[k] = make_float2(-INFINITY, 0.f);
        if (!there || !mine) return;
        ml[k] = p.part_ml[at * kTileRows + row];
#pragma unroll
        for (int x = 0; x < kJoinDims / 4; ++x)
            v[k][x] = reinterpret_cast<const float4 *>(p.part_o)[at * (D / 4 * kTileRows) + (d0 / 4 + x) * kTileRows + row];
    };
    auto merge = [&](int k) {
        if (ml[k].y == 0.f) return;  // saw nothing there
        const float to = fmaxf(m, ml[k].x), a = m == -INFINITY ? 0.f : exp2f(m - to), b = ml[k].x == -INFINITY ? 1.f : exp2f(ml[k].x - to);
        m = to;
        l = l * a + ml[k].y * b;
#pragma unroll
        for (int x = 0; x < kJoinDims / 4; ++x)
            o[x] = make_float4(o[x].x * a + v[k][x].x * b, o[x].y * a + v[k][x].y * b, o[x].z * a + v[k][x].z * b, o[x].w * a + v[k][x].w * b);
    };
    fetch(0, 2 * w + 1, true);
    merge(0);
    // the workers after it, 32 at a time: those that have a part, up to the one with the unit's end
    const int lane = threadIdx.x & 31;
    for (int u0 = w + 1; u0 < p.workers; u0 += 32) {
        const int head = u0 + lane < p.workers ? p.meta[u0 + lane].head : 0;
        const uint32_t ends = __ballot_sync(0xffffffffu, head <= 1), until = ends ? __ffs(ends) - 1 : 31;
        uint32_t parts = __ballot_sync(0xffffffffu, head == 1 || head == 2) & (0xffffffffu >> (31 - until));
        while (parts) {
#pragma unroll
            for (int k = 0; k < kJoinAtOnce; ++k) {
                const int at = __ffs(parts) - 1;
                fetch(k, 2 * (u0 + (at < 0 ? 0 : at)), at >= 0);
                parts &= parts - 1;
            }
#pragma unroll
            for (int k = 0; k < kJoinAtOnce; ++k) merge(k);
        }
        if (ends) break;
    }
    if (!mine) return;
    const int64_t trow = meta.row0 + tok;
    const int hq = meta.h * p.G + row % p.G;
    const float inv = 1.f / l;
    uint32_t r[kJoinDims / 2];
#pragma unroll
    for (int x = 0; x < kJoinDims / 4; ++x) {
        const float4 y = l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o[x].x * inv, o[x].y * inv, o[x].z * inv, o[x].w * inv);
        r[2 * x] = p.bf16 ? pack<true>(y.x, y.y) : pack<false>(y.x, y.y);
        r[2 * x + 1] = p.bf16 ? pack<true>(y.z, y.w) : pack<false>(y.z, y.w);
    }
    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + (trow * p.out_stride + (int64_t)hq * D + d0));
#pragma unroll
    for (int x = 0; x < kJoinDims / 8; ++x) dst[x] = make_uint4(r[4 * x], r[4 * x + 1], r[4 * x + 2], r[4 * x + 3]);
    if (d0 == 0 && p.lse) p.lse[trow * p.Hq + hq] = l == 0.f ? -INFINITY : (m + log2f(l) - kUp) * 0.693147180559945309f;
}

// ---------------------------------------------------------------- host side

kvs_status bad(kvs_status s, const char *why) {
    set_thread_error(why);
    return s;
}
kvs_status cuda_failed(const char *what, cudaError_t e) {
    cudaGetLastError();  // the call's own: no later one is to find it
    set_thread_error(std::string(what) + ": " + cudaGetErrorString(e));
    return KVS_ERR_CUDA;
}
bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

uint64_t part_rows(uint32_t D) { return 2ull * kWorkers * (D <= 128 ? 2 : 1) * kTileRows; }
uint64_t workspace_of(uint32_t D) { return (part_rows(D) * (D * 4 + 8) + kWorkers * sizeof(ChunkMeta) + 255) / 256 * 256; }

template <int D>
kvs_status launch_chunk(const ChunkParams &p, cudaStream_t s) {
    using S = ChunkShape<D>;
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(chunk_kernel<D>), S::kSmem);
    if (e != cudaSuccess) return cuda_failed("chunk attention launch", e);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.workers);
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = s;
    e = cudaLaunchKernelEx(&cfg, chunk_kernel<D>, p);
    if (e != cudaSuccess) return cuda_failed("chunk attention launch", e);
    cfg.gridDim = dim3((unsigned)p.workers, S::NQ * D / kJoinDims);
    cfg.blockDim = dim3(kTileRows);
    cfg.dynamicSmemBytes = 0;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, join_kernel<D>, p);
    return e == cudaSuccess ? KVS_OK : cuda_failed("chunk join launch", e);
}

}  // namespace
}  // namespace kvs

using namespace kvs;

extern "C" kvs_status kvs_q4_chunk_workspace(const kvs_q4_pool *pool, uint64_t *workspace_bytes) {
    Q4Pool p = {};
    const kvs_status s = check_q4_pool(pool, false, &p);
    if (s != KVS_OK) return s;
    if (!workspace_bytes) return bad(KVS_ERR_INVALID, "null workspace_bytes");
    *workspace_bytes = workspace_of(pool->head_dim);
    return KVS_OK;
}

extern "C" kvs_status kvs_q4_attend_chunk(const kvs_q4_pool *pool, const int32_t *table, uint32_t table_width, const int32_t *lens,
                                          const int32_t *cu, uint32_t n_seq, uint32_t total_rows, uint32_t n_q_head, const void *q,
                                          int32_t dtype, uint64_t q_stride, float scale, uint32_t window, uint32_t sinks, void *out,
                                          uint64_t out_stride, float *lse, void *workspace, uint64_t workspace_bytes, void *stream) {
    ChunkParams p = {};
    kvs_status s = check_q4_pool(pool, true, &p.pool);
    if (s != KVS_OK) return s;
    if (dtype == KVS_F32) return bad(KVS_ERR_UNSUPPORTED, "chunks are KVS_F16 or KVS_BF16");
    if (dtype != KVS_F16 && dtype != KVS_BF16) return bad(KVS_ERR_INVALID, "dtype must be KVS_F16 or KVS_BF16");
    const uint32_t D = pool->head_dim, Hk = pool->n_kv_head;
    if (n_q_head < Hk || n_q_head % Hk != 0 || n_q_head > 65535)
        return bad(KVS_ERR_INVALID, "n_q_head must be a positive multiple of n_kv_head, at most 65535");
    if (n_q_head / Hk > (uint32_t)kMaxGroup) return bad(KVS_ERR_UNSUPPORTED, "n_q_head / n_kv_head must be at most 64");
    if (n_seq > (uint32_t)kMaxSeq) return bad(KVS_ERR_UNSUPPORTED, "n_seq must be at most 4096");
    if (total_rows > 0x7fffffffu - 256u) return bad(KVS_ERR_INVALID, "total_rows must be at most 2^31 - 1 - 256");
    if (table_width < 1 || (uint64_t)table_width * pool->page_tokens > 0x7fffffc0ull)
        return bad(KVS_ERR_INVALID, "table_width * page_tokens must be 1 .. 2^31 - 64");
    if (!isfinite(scale)) return bad(KVS_ERR_INVALID, "scale must be finite");
    if (window > 0x7fffffffu || sinks > 0x7fffffffu - 64u) return bad(KVS_ERR_INVALID, "window and sinks must be at most 2^31 - 65");
    if (n_seq && (!table || !lens || !cu)) return bad(KVS_ERR_INVALID, "null table, lens or cu");
    const uint64_t row = (uint64_t)n_q_head * D;
    if (n_seq && total_rows) {
        if (!q || !out) return bad(KVS_ERR_INVALID, "null q or out");
        if (!aligned(q, 16) || !aligned(out, 16) || q_stride % 8 || out_stride % 8 || q_stride < row || out_stride < row)
            return bad(KVS_ERR_INVALID, "rows must start on 16-byte boundaries, at least n_q_head * head_dim apart");
        if (q_stride > (1ull << 31) || out_stride > (1ull << 31)) return bad(KVS_ERR_INVALID, "row stride too large");
        if (!workspace || !aligned(workspace, 256)) return bad(KVS_ERR_INVALID, "workspace null or not 256-byte aligned");
        if (workspace_bytes < workspace_of(D)) return bad(KVS_ERR_CAPACITY, "workspace smaller than kvs_q4_chunk_workspace asks for");
    }
    if (n_seq == 0 || total_rows == 0) return KVS_OK;
    const int sms = current_device_sms();
    const uint32_t fault = batch_fault();
    p.give_up = fault == KVS_FAULT_DEVICE_WAIT;
    p.late = fault == KVS_FAULT_DEVICE_LATE;
    p.table = table;
    p.lens = lens;
    p.cu = cu;
    p.table_width = (int)table_width;
    p.n_seq = (int)n_seq;
    p.total = (int)total_rows;
    p.Hq = (int)n_q_head;
    p.G = (int)(n_q_head / Hk);
    p.workers = sms < kWorkers ? sms : kWorkers;
    const bool windowed = window > 0 && window < (uint64_t)table_width * pool->page_tokens;  // (else every token is inside)
    p.window = windowed ? (int)window : 0;
    p.sinks = windowed ? (int)sinks : 0;
    p.q = q;
    p.q_stride = (int64_t)q_stride;
    p.bf16 = dtype == KVS_BF16;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.out = out;
    p.out_stride = (int64_t)out_stride;
    p.lse = lse;
    p.part_o = static_cast<float *>(workspace);
    p.part_ml = reinterpret_cast<float2 *>(p.part_o + part_rows(D) * D);
    p.meta = reinterpret_cast<ChunkMeta *>(p.part_ml + part_rows(D));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return D == 64 ? launch_chunk<64>(p, st) : D == 128 ? launch_chunk<128>(p, st) : launch_chunk<256>(p, st);
}
