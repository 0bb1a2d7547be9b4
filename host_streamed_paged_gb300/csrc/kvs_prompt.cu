// Attention over packed prompts, and the attention weight that their keys
// receive, on the 5th-generation tensor cores (include/kvs.h, kvs_prompt_*).
//
// Rows.  A kv head's query rows are its tokens' G query heads, token by token:
// a 128-row MMA tile holds floor(128 / G) tokens of all G heads, read by one
// TMA box.  So K and V are read once per kv head, short prompts fill tiles,
// and the causal edge of a tile spans 128 / G keys instead of 128.
//
// Windows.  A unit walks the key blocks of the first tokens, then those from its
// first row's window on; a block's index is all that knows of the gap between
// them.  Units are short then and all alike, so one CTA per SM takes every
// gridDim.x-th of them: the next one's Q comes in once the last S is done, its
// first scores are formed under the last one's P V and output (16755 rows of 8192
// + 6001 + 2048 + 513 + 1 tokens, window 1024, 32 / 8 heads, D 128, bf16: 280 us
// with a CTA a unit, 262 so, 255 with the next unit found while the last P V is
// under way; 0.98 PFLOP/s of seen pairs).  A block of both tiles takes 0.74 us,
// which is the tensor pipe's pace, a unit's change 6 us beside 18 blocks.  (Found
// earlier, between blocks, 273; outputs turned around among four lanes, so that
// a store is of fewer lines, 264.)  Over more
// than 256 prompts a warp goes through them once, not once a unit: 4096 prompts
// of 70 tokens, window 50, 12.9 -> 2.5 ms.  The kernels without a window are
// compiled apart and hold none of it.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include <mutex>
#include <string>

#include "kvs.h"
#include "kvs_internal.h"
#include "kvs_tcgen05.cuh"

namespace kvs {
namespace {

namespace cg = cooperative_groups;
using namespace tc;

constexpr int kThreads = 384;  // warps 0-3, 4-7: one softmax warpgroup per tile; warp 8: MMA issue; warp 9: TMA
constexpr int kMaxSeq = 4096;
constexpr int kMaxGroup = 64;

// ---------------------------------------------------------------- which prompt, which tile

struct PromptParams {
    const int32_t *cu;
    int n_seq, total, Hk, G;
    float scale_log2;
    void *out;
    int64_t out_stride;
    float *lse;
    // weights
    const float *lse_in;
    const float *prev;
    float *w;
    int64_t width;
    int last_rows;
    int window, sinks, units;  // of the windowed kernels; units: bound of (tile groups x heads)
    int main_ctas;  // those past them copy what no key writes
    int give_up;    // test hook: the MMA warps give up at their first wait, as if its copy never landed, and *abort is up
    int late;       // test hook (windows): the one of a tile with a block at most comes late to the unit's second
};

__device__ __forceinline__ int cu_begin(const PromptParams &p, int s) {
    const int a = p.cu[s];
    return a < 0 ? 0 : (a < p.total ? a : p.total);
}
__device__ __forceinline__ int cu_end(const PromptParams &p, int s) {
    const int a = cu_begin(p, s), b = p.cu[s + 1];
    return b < a ? a : (b < p.total ? b : p.total);
}

// Where unit `c` of the launch lies: prompt s, group x of its `per`-token groups
// counted so that a larger x is more work (place = {s, x, begin, end, groups};
// s < 0 past the last).  Units go out heaviest first over all prompts, since a
// causal tile's work grows with x and a heavy one begun late would run alone
// at the end: level by level from the longest prompt's last group down.  (Up
// to 256 prompts, which a warp holds in registers; of more prompts each is a
// small part of the launch and they go one after another.)  Called by a warp,
// before anything else of a CTA can begin, so kept short: one round of loads and
// few instructions (some 1000 clocks; 3000 with 256 prompts' registers always).
constexpr int kSortedSeq = 256;
template <int kEach>
__device__ __forceinline__ void find_sorted(const PromptParams &p, int c, int per, int *place) {
    const int lane = threadIdx.x & 31;
    int from_[kEach], to[kEach], t[kEach], most = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int s = 32 * i + lane;
        from_[i] = s < p.n_seq ? p.cu[s] : 0;
        to[i] = s < p.n_seq ? p.cu[s + 1] : 0;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        from_[i] = max(0, min(from_[i], p.total));
        to[i] = max(from_[i], min(to[i], p.total));
        t[i] = (to[i] - from_[i] + per - 1) / per;
        most = max(most, t[i]);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    auto units = [&](int level) {  // at this level or above (per prompt max(0, t - level))
        int n = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) n += max(0, t[i] - level);
        return __reduce_add_sync(0xffffffffu, n);
    };
    int lo = 0, hi = most - 1, above = 0;  // the largest level with c < units(level); above: units(lo + 1) at the end
    if (lane == 0) place[0] = -1;
    __syncwarp();
    if (c >= units(0)) return;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1, n = units(mid);
        if (c < n) lo = mid;
        else hi = mid - 1, above = n;
    }
    int nth = c - above;  // among the prompts with a group at this level
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const uint32_t has = __ballot_sync(0xffffffffu, t[i] > lo);
        const int n = __popc(has);
        if (nth >= 0 && nth < n && __popc(has & ((1u << lane) - 1)) == nth && (has >> lane & 1)) {
            place[0] = 32 * i + lane;
            place[1] = lo;
            place[2] = from_[i];
            place[3] = to[i];
            place[4] = t[i];
        }
        nth -= n;
    }
}
// RESUME: of ascending c; place[6] and [7], 0 at first, hold how far the prompts
// were gone through (from the first on each time, 4096 prompts take a unit 25 us).
template <bool RESUME = false>
__device__ __forceinline__ void find_unit(const PromptParams &p, int c, int per, int *place) {
    const int lane = threadIdx.x & 31;
    if (p.n_seq <= 32) return find_sorted<1>(p, c, per, place);
    if (p.n_seq <= kSortedSeq) return find_sorted<kSortedSeq / 32>(p, c, per, place);
    auto groups = [&](int s) { return s < p.n_seq ? (cu_end(p, s) - cu_begin(p, s) + per - 1) / per : 0; };
    int s = -1, x = 0, base = RESUME ? place[7] : 0, s0 = RESUME ? place[6] : 0;
    for (; s0 < p.n_seq; s0 += 32) {
        const int t = groups(s0 + lane);
        int inc = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, base + inc > c);
        if (past) {
            const int who = __ffs(past) - 1;
            s = s0 + who;
            x = __shfl_sync(0xffffffffu, base + inc, who) - 1 - c;
            break;
        }
        base += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (RESUME) {
        __syncwarp();
        if (lane == 0) place[6] = s0, place[7] = base;
    }
    if (lane == 0) {
        place[0] = s;
        if (s >= 0) {
            place[1] = x;
            place[2] = cu_begin(p, s);
            place[3] = cu_end(p, s);
            place[4] = groups(s);
        }
    }
}

// ---------------------------------------------------------------- attention
// Per CTA and kv head: two 128-row query tiles (D <= 128) or one (D = 256: its
// O takes the tensor memory of two) against the prompt's key blocks.
//   warp 9 loads Q, then K and V through a ring (TMA);
//   warp 8 + 2 i issues tile i's S = Q K^T into tensor memory and O += P V, P as
//     the tensor-memory A operand over S's columns (one issuing warp per tile:
//     a warp's MMAs leave it only as the pipe takes them, and it then needs
//     200 clocks to see the next barrier; two warps fill each other's gaps);
//   each softmax warpgroup (one thread per row) turns its tile's S into P and
//     rescales O only when a row's maximum grew by more than 2^8.
// Each tile has two score buffers and its S runs two blocks ahead, so that a
// warpgroup finds the next scores ready when it is done with the last and the
// tensor pipe never waits for a softmax.  Tensor memory (512 columns) then
// allows blocks of 64 keys for two tiles, and 128 for the one of D = 256.  An
// S MMA of N = 64 takes 50 clocks for 2/3 of the work of one of N = 128 (66
// clocks: it reads its A tile from shared memory anew), which costs less than
// the one 128-key buffer per tile that would fit: its softmax waits for its
// own P V and Q K^T each time.
// The tensor pipe bounds long prompts: 16755 rows of prompts of 8192 .. 1
// tokens, 32 / 8 heads, D 128, bf16, take 577 us, 1.53 PFLOP/s of causal work
// (79% of the measured bf16 rate; 600 to 620 in a long run, under the power
// cap; a third longer with one issuing warp and S one block ahead).  8192 +
// 6001 tokens, 24 / 4 heads, D 256: 1310 us, 0.97 PFLOP/s, bound by K and V
// through L2, 128 KB per 128 keys for one tile.  Short prompts take a CTA's
// chain of starts and waits: five of 1 .. 300 tokens, 24 / 4 heads, D 256, 16
// us, as long as the rate allows 3 us.
template <int D>
struct AttendShape {
    static constexpr int NQ = D <= 128 ? 2 : 1;
    static constexpr int BN = D <= 128 ? 64 : 128;
    static constexpr int kQBytes = kTileRows * D * 2;
    static constexpr int kPieces = D == 256 ? 4 : 1;  // ring stages of a block: K by 64 dims (D = 256), V by keys
    static constexpr int kPiece = BN * D * 2 / kPieces;
    static constexpr int kVKeys = BN / kPieces;       // keys of a V piece
    static constexpr int kStages = D == 64 ? 12 : 10;
    static constexpr int kOffRing = NQ * kQBytes;
    static constexpr int kOffBar = kOffRing + kStages * kPiece;
    static constexpr int kSmem = kOffBar + 1024 + 1024;
    static constexpr uint32_t kColO = 256;
};

template <int D, bool BF16, bool WIN>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attend_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ CUtensorMap mq,
                         const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    using S = AttendShape<D>;
    constexpr int NQ = S::NQ, BN = S::BN, NST = S::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t bars = smem_u32(smem + S::kOffBar);
    // barriers: ring full / empty, Q full, final; per tile and score buffer: S full, P full, O done (by the same parity); Q
    // read by all its MMAs
    auto b_full = [&](int s) { return bars + 8u * s; };
    auto b_empty = [&](int s) { return bars + 8u * (12 + s); };
    const uint32_t b_q = bars + 8u * 24, b_final = bars + 8u * 25;
    auto b_s = [&](int i, int buf) { return bars + 8u * (26 + 2 * i + buf); };
    auto b_p = [&](int i, int buf) { return bars + 8u * (30 + 2 * i + buf); };
    auto b_o = [&](int i, int buf) { return bars + 8u * (34 + 2 * i + buf); };
    const uint32_t b_q_read = bars + 8u * 38;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::kOffBar + 8 * 39);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + S::kOffBar + 8 * 40);
    int *place = reinterpret_cast<int *>(smem + S::kOffBar + 8 * 41);  // the first unit; [8 (1 + warp)]: a warp's next one

    const int G = p.G, TQ = kTileRows / G;
    int unit = blockIdx.x, head = unit % p.Hk;
    // the work is found, tensor memory allocated and the barriers set up by three warps at once
    if (warp == 9) find_unit(p, blockIdx.x / p.Hk, NQ * TQ, place);
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid == 32) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(b_full(s), 1);
            mbar_init(b_empty(s), NQ);
        }
        mbar_init(b_q, 1);
        mbar_init(b_final, NQ);
        if (WIN) mbar_init(b_q_read, NQ);
        for (int i = 0; i < 4; ++i) {
            mbar_init(b_s(0, i), 1);
            mbar_init(b_p(0, i), 4);
            mbar_init(b_o(0, i), 1);
        }
        *abort = p.give_up;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = *tmem_slot;
    if (place[0] < 0) {
        if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
        return;
    }
    int begin, L, t0;  // of the unit: its prompt's first row and length, tile 0's first token within the prompt
    // under a window the blocks of the first tokens, `front` of them, then those from the first row's window on: block j is
    // j, or j + skip from `front` on
    int front = 0, skip = 0, nblk[2] = {0, 0}, n_max;
    auto key_block = [&](int j) { return WIN && j >= front ? j + skip : j; };
    auto set_unit = [&](const int *at) {
        begin = at[2], L = at[3] - begin;
        t0 = at[1] * NQ * TQ;
        if constexpr (WIN) {
            const int first = t0 >= p.window ? (t0 - p.window + 1) / BN : 0;
            front = min((p.sinks + BN - 1) / BN, first);
            skip = first - front;
        }
        n_max = 0;
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            const int a = t0 + i * TQ, last = (a + TQ < L ? a + TQ : L) - 1;
            nblk[i] = a < L ? last / BN + 1 - skip : 0;
            n_max = nblk[i] > n_max ? nblk[i] : n_max;
        }
    };
    set_unit(place);
    if (WIN && lane < 2) place[8 * (1 + warp) + 6 + lane] = 0;
    // Under a window a CTA takes every gridDim.x-th unit, each warp finding them by itself; what it counts over them:
    // units, ring stages, blocks of its tile (0 all along in the kernels of one unit)
    int nth = 0, ring0 = 0, blk0 = 0;
    auto next_unit = [&] {
        if constexpr (WIN) {
            ring0 += 2 * n_max * S::kPieces;
            ++nth;
            unit += gridDim.x;
            if (unit >= p.units) return false;
            int *at = place + 8 * (1 + warp);
            __syncwarp();
            find_unit<true>(p, unit / p.Hk, NQ * TQ, at);
            __syncwarp();
            if (at[0] < 0) return false;
            head = unit % p.Hk;
            set_unit(at);
            return true;
        }
        return false;
    };
    // the ring's blocks in the order the MMAs take them: K_0, K_1, V_0, K_2, V_1, ..., K_{n-1}, V_{n-2}, V_{n-1},
    // kPieces stages each
    auto ring_k = [&](int j) { return ring0 + (j < 2 ? j : 2 * j - 1) * S::kPieces; };
    auto ring_v = [&](int j) { return ring0 + (j == n_max - 1 ? 2 * n_max - 1 : 2 * j + 2) * S::kPieces; };
    auto load_piece = [&](int r) {
        const int st = (ring0 + r) % NST, q = r / S::kPieces, c = r % S::kPieces, end = 2 * n_max - 1;
        const bool is_v = q == end || (q >= 2 && !(q & 1));
        const int j = key_block(q == end ? n_max - 1 : (q < 2 ? q : (q & 1 ? (q + 1) / 2 : q / 2 - 1)));
        const uint32_t dst = smem_u32(smem + S::kOffRing + st * S::kPiece);
        mbar_expect(b_full(st), (uint32_t)S::kPiece);
        if (is_v) {
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
                tma_load(dst + x * S::kVKeys * 128, &mv, b_full(st), x * 64, head, begin + j * BN + c * S::kVKeys);
        } else {
#pragma unroll
            for (int x = 0; x < D / 64 / S::kPieces; ++x)
                tma_load(dst + x * BN * 128, &mk, b_full(st), (c + x) * 64, head, begin + j * BN);
        }
    };
    if (warp == 9) {
        // ------------------------------------------------------------ loads
        int issued = 0;
        bool ok = true;
        do {
            if (lane == 0) {
                if (WIN && nth > 0) ok = mbar_wait(b_q_read, (uint32_t)((nth - 1) & 1), abort);
                if (ok) {
                    place[6] = nth;
                    mbar_expect(b_q, (uint32_t)(NQ * (D / 64) * 128 * G * TQ));
                    for (int i = 0; i < NQ; ++i)
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            tma_load(smem_u32(smem + i * S::kQBytes + c * kTileRows * 128), &mq, b_q, c * 64, head * G, begin + t0 + i * TQ);
                }
                const int n_ring = 2 * n_max * S::kPieces;
                for (int r = 0; r < n_ring && ok; ++r) {
                    const int at = ring0 + r;
                    if (at >= NST && !mbar_wait(b_empty(at % NST), (uint32_t)((at / NST - 1) & 1), abort)) {
                        ok = false;
                        break;
                    }
                    load_piece(r);
                    issued = at + 1;
                }
            }
        } while (WIN && __shfl_sync(0xffffffffu, ok, 0) && next_unit());
        if (lane == 0) place[5] = issued;
    } else if (warp == 8 || (NQ == 2 && warp == 10)) {
        const int i = (warp - 8) >> 1;
        int n = nblk[i];
        // ------------------------------------------------------------ MMA issue (the warp in step, one elected lane issues)
        constexpr uint32_t id_s = idesc(BF16, kTileRows, BN, false), id_o = idesc(BF16, kTileRows, D, true);
        constexpr int NP = S::kPieces;
        const bool one = elect_one();
        const uint64_t dq = smem_desc(smem_u32(smem), 16), dk = smem_desc(smem_u32(smem + S::kOffRing), 16);
        const uint64_t dv = smem_desc(smem_u32(smem + S::kOffRing), S::kVKeys * 128);
        auto stage = [&](int r, int c) { return (r + c) % NST; };
        auto loaded = [&](int r) {  // a block's pieces
            bool all = true;
#pragma unroll
            for (int c = 0; c < NP; ++c) all &= mbar_done(b_full(stage(r, c)), (uint32_t)(((r + c) / NST) & 1));
            return all;
        };
        auto freed = [&](int r) {
#pragma unroll
            for (int c = 0; c < NP; ++c) mma_commit(b_empty(stage(r, c)));
        };
        auto issue_s = [&](int j) {
            const uint32_t d = tmem + (uint32_t)((2 * i + ((blk0 + j) & 1)) * BN);
            const uint64_t da = dq + (uint64_t)(i * S::kQBytes >> 4);
            const int r = ring_k(j);
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                constexpr int kPer = D / 16 / NP;  // 16-dim steps of a piece
                const uint64_t db = dk + (uint64_t)((stage(r, s / kPer) * S::kPiece + (s % kPer >> 2) * (BN * 128) + (s & 3) * 32) >> 4);
                mma_ss(d, da + (uint64_t)(((s >> 2) * (kTileRows * 128) + (s & 3) * 32) >> 4), db, id_s, s > 0);
                if (s % kPer == kPer - 1) mma_commit(b_empty(stage(r, s / kPer)));  // its loads need not wait for the rest
            }
            mma_commit(b_s(i, (blk0 + j) & 1));
            if (WIN && j == n - 1) mma_commit(b_q_read);
        };
        auto issue_o = [&](int j) {
            const uint32_t d = tmem + S::kColO + (uint32_t)(i * D), a = tmem + (uint32_t)((2 * i + ((blk0 + j) & 1)) * BN);
            const int r = ring_v(j);
#pragma unroll
            for (int s = 0; s < BN / 16; ++s) {
                constexpr int kPer = BN / 16 / NP;  // 16-key steps of a piece
                const uint64_t db = dv + (uint64_t)((stage(r, s / kPer) * S::kPiece + s % kPer * 2048) >> 4);
                mma_ts(d, a + (uint32_t)(8 * s), db, id_o, (j > 0 || s > 0) ? 1u : 0u);
                if (s % kPer == kPer - 1) mma_commit(b_empty(stage(r, s / kPer)));
            }
            mma_commit(b_o(i, (blk0 + j) & 1));
        };
        // a block past this tile's last one is freed as it comes, for the other tile's sake
        bool ok = !p.give_up;
        do {
            n = nblk[i];
            for (int j = 0; j < 2 && j < n_max && ok; ++j) {
                if (WIN && p.late && j == 1 && n < 2)
                    for (int k = 0; k < 50; ++k) __nanosleep(1000);
                // (Q is asked for at the first block alone: a tile of no more blocks gives it back there, and once the next
                // unit's has come this phase would not be seen any more)
                ok = wait_warp(abort, [&] { return (j > 0 || mbar_done(b_q, (uint32_t)(nth & 1))) & loaded(ring_k(j)); });
                if (!ok) break;
                tc_after();
                if (one) {
                    if (j < n) issue_s(j);
                    else freed(ring_k(j));
                    if (WIN && j == 0 && n == 0) mma_commit(b_q_read);  // (not before its Q has come: an earlier phase may be open)
                }
            }
            // S_{j+2} takes the buffer of S_j and P_j: P_j was read by O's MMA before it, and the pipe keeps their order
            for (int j = 0; j < n_max && ok; ++j) {
                const bool more = j + 2 < n_max;
                ok = wait_warp(abort, [&] {
                    bool all = loaded(ring_v(j));
                    if (j < n) all &= mbar_done(b_p(i, (blk0 + j) & 1), (uint32_t)(((blk0 + j) >> 1) & 1));
                    if (more) all &= loaded(ring_k(j + 2));
                    return all;
                });
                if (!ok) break;
                tc_after();
                if (one) {
                    if (j < n) issue_o(j);
                    else freed(ring_v(j));
                    if (j + 2 < n) issue_s(j + 2);
                    else if (more) freed(ring_k(j + 2));
                }
            }
            blk0 += n;
        } while (ok && next_unit());
        if (one) mma_commit(b_final);  // on every path: tensor memory is freed only after it
    } else if (warp < 4 * NQ) {
        // ------------------------------------------------------------ softmax, one thread per row
        const int i = warp >> 2, row = tid & 127;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const float sc = p.scale_log2;
        // P is 2^(s - m + kUp), at most 2^(8 + kUp): as high as f16 reaches, so that its smallest step is 2^-31 of the largest
        // weight or less (2^-24 without, and thousands of keys below it are lost from the output); bf16 has the exponents
        constexpr float kUp = BF16 ? 0.f : 7.f;
        bool ok = true, more;
        do {
            const int n = nblk[i], tok = t0 + i * TQ + row / G;  // within the prompt
            const bool valid = row < TQ * G && tok < L;
            float m = -INFINITY;
            float2 l2 = make_float2(0.f, 0.f);
            const int first_tok = t0 + i * TQ;
            for (int j = 0; (!WIN || ok) && j < n; ++j) {
                const int buf = (blk0 + j) & 1;
                ok = mbar_wait_warp(b_s(i, buf), (uint32_t)(((blk0 + j) >> 1) & 1), abort);
                if (!ok) break;
                tc_after();
                const uint32_t ts = lanes + (uint32_t)((2 * i + buf) * BN);
                uint32_t sr[BN];
#pragma unroll
                for (int c = 0; c < BN; c += 32) tmem_ld32(ts + c, sr + c);
                tmem_wait_ld();
                float *s = reinterpret_cast<float *>(sr);
                const int kb = key_block(j);
                if ((kb + 1) * BN > first_tok + 1) {  // some row of the tile ends inside the block
                    const int lim = tok - kb * BN;
#pragma unroll
                    for (int c = 0; c < BN; ++c) s[c] = c <= lim ? s[c] : -INFINITY;
                }
                if constexpr (WIN) {
                    // some row's window begins behind the block's first key, and not all of its keys are of the first that stay
                    if (kb * BN <= first_tok + TQ - 1 - p.window && (kb + 1) * BN > p.sinks) {
                        const int from = tok - p.window - kb * BN, stay = p.sinks - kb * BN;
#pragma unroll
                        for (int c = 0; c < BN; ++c) s[c] = c > from || c < stay ? s[c] : -INFINITY;
                    }
                }
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < BN; c += 2) m4[(c >> 1) & 3] = fmax3(m4[(c >> 1) & 3], s[c], s[c + 1]);
                const float mx = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]) * sc;
                const bool grow = mx > m + 8.f || (m == -INFINITY && mx != -INFINITY);
                if (__any_sync(0xffffffffu, grow)) {
                    const float to = grow ? mx : m;
                    const float alpha = m == -INFINITY ? 0.f : ex2(m - to);
                    l2.x *= alpha;
                    l2.y *= alpha;
                    m = to;
                    if (j > 0) {
                        ok = mbar_wait_warp(b_o(i, (blk0 + j - 1) & 1), (uint32_t)(((blk0 + j - 1) >> 1) & 1), abort);
                        if (!ok) break;
                        tc_after();
                        const uint32_t to_o = lanes + S::kColO + (uint32_t)(i * D);
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t v[32];
                            tmem_ld32(to_o + c, v);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
                            tmem_st32(to_o + c, v);
                        }
                    }
                }
                const float neg = m == -INFINITY ? 0.f : kUp - m;
                const float2 sc2 = make_float2(sc, sc), neg2 = make_float2(neg, neg);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int part = 0; part < BN / 64; ++part) {
                    uint32_t pk[32];
#pragma unroll
                    for (int c = 0; c < 64; c += 2) {
                        const float2 y = fma2(make_float2(s[64 * part + c], s[64 * part + c + 1]), sc2, neg2);
                        const float2 e = make_float2(ex2(y.x), ex2(y.y));
                        sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], e);
                        pk[c / 2] = pack<BF16>(e.x, e.y);
                    }
                    tmem_st32(ts + 32 * part, pk);
                }
                l2 = add2(l2, add2(sum[0], sum[1]));
                if ((kb + 1) * BN > L) {
                    // the block reaches past the prompt: its last rows are another prompt's (or nobody's), and a weight
                    // of zero times what stands there must be zero
#pragma unroll
                    for (int c = 0; c < S::kPieces; ++c) {
                        const int r = ring_v(j) + c, st = r % NST;
                        ok = ok && mbar_wait_warp(b_full(st), (uint32_t)((r / NST) & 1), abort);
                        if (ok && row < S::kVKeys && kb * BN + c * S::kVKeys + row >= L) {
#pragma unroll
                            for (int x = 0; x < D / 64; ++x)
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    *reinterpret_cast<uint4 *>(smem + S::kOffRing + st * S::kPiece + (x * S::kVKeys + row) * 128 + k * 16) =
                                        make_uint4(0, 0, 0, 0);
                        }
                    }
                    proxy_fence();
                }
                tmem_wait_st();
                if (!ok) break;
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_p(i, buf));
            }
            const int last = blk0 + n - 1;
            const int64_t trow = begin + tok;
            const int hq = head * G + row % G;
            blk0 += n;
            more = next_unit();  // while the last P V is under way
            if (ok && n > 0) ok = mbar_wait_warp(b_o(i, last & 1), (uint32_t)((last >> 1) & 1), abort);
            if (n > 0) {
                tc_after();
                const float l = l2.x + l2.y;
                const float inv = ok ? 1.f / l : __int_as_float(0x7fc00000);
                const uint32_t to = lanes + S::kColO + (uint32_t)(i * D);
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + (trow * p.out_stride + (int64_t)hq * D));
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t v[32] = {};
                    if (ok) {  // (the same in a warp; else MMAs may be under way, and what they have is not wanted)
                        tmem_ld32(to + c, v);
                        tmem_wait_ld();
                    }
                    if (valid) {
#pragma unroll
                        for (int k = 0; k < 32; k += 8) {
                            uint32_t o[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                o[x] = pack<BF16>(__uint_as_float(v[k + 2 * x]) * inv, __uint_as_float(v[k + 2 * x + 1]) * inv);
                            dst[(c + k) / 8] = make_uint4(o[0], o[1], o[2], o[3]);
                        }
                    }
                }
                if (valid && p.lse)
                    p.lse[trow * (int64_t)(p.Hk * G) + hq] = ok ? (m + log2f(l * (BF16 ? 1.f : 0.0078125f))) * 0.693147180559945309f : inv;
            }
        } while (more);
    }
    // tensor memory is freed once every MMA is done and every row was read
    if (tid == 0) mbar_drain(b_final, 0);
    tc_before();
    __syncthreads();
    tc_after();
    // Every role is done.  If one gave up, copies that no one waited for may still be under way into this CTA's shared
    // memory, which is its own while this lane stays.  (Otherwise the MMAs have waited for all of them.)
    if (tid == 9 * 32 && *abort) {
        const int issued = place[5];
        mbar_drain(b_q, (uint32_t)(place[6] & 1));
        for (int st = 0; st < NST; ++st)
            if (issued > st) mbar_drain(b_full(st), (uint32_t)(((issued - 1 - st) / NST) & 1));
    }
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ---------------------------------------------------------------- weights
// w_j = sum over rows of exp(s_ij - lse_i).  Keys are the M rows here, so a
// thread owns one key: S^T = K Q^T, a 128-key tile per CTA against a stream of
// query tiles, each read from tensor memory once, exponentiated against the
// rows' lse and added up in a register.  Two warpgroups share the tile, half of
// the columns each.  Two CTAs fit an SM, so that one's start, end and waits
// pass under the other's work.  What bounds it is a sum warp's chain (scores
// from tensor memory, multiply-add, exponential, add): 1450 clocks of an SM for
// 128 x 128 scores, of which the exponentials are 512 (32 a clock) and the MMAs
// 530 at D = 128.  The first keys of a prompt are seen by all its rows; so that
// such a unit does not hold up the launch, a cluster shares it, every CTA a
// part of the query tiles, and adds its sums up in rank order.
// At D = 256 a tile is 96 rows: K leaves the ring of two CTAs 36 KB, which are
// two stages of 128 rows, and 64 rows pay the 50-clock MMA of N = 64 (52 us on
// the window below, 46 with 96).  Its scores are summed over 128 dims each, in
// two accumulators: the tensor core drops what lies below an accumulator's last
// place at every 16 dims, always towards zero, and with 256 dims in a row the
// weights came out 1.1e-6 low, 6e-7 like this (4 us more).
// Prompts of 4096 .. 33 tokens, 32 / 8 heads, D 128, over all rows: 114 us (121
// with the causal edge's test among the columns of every tile; a quarter longer
// with two key tiles in one CTA of 16 sum warps, up to a half with 2 to all of
// 16 exponentials of those as polynomials on the FMA pipes).  The last 64 rows
// of 32768, 24 / 4 heads, D 256: 40 to 45 us a call, 48 with a cold cache.
constexpr int kWThreads = 320;  // warps 0-7: sums; 8: MMA issue; 9: TMA
template <int D>
struct WeightShape {
    static constexpr int BQ = D <= 128 ? 128 : 96;  // query rows per tile
    static constexpr int kCols = BQ / 2;            // of them a warpgroup's
    static constexpr int kChunks = D / 64;          // a tile's ring stages: 64 dims each
    static constexpr int kStep = D == 128 ? 2 : 1;  // stages waited for at once
    static constexpr int kKBytes = kTileRows * D * 2;
    static constexpr int kChunk = BQ * 128;
    static constexpr int kStages = D == 256 ? 3 : 4;
    static constexpr int kParts = D == 256 ? 2 : 1;    // sums of a score: over 128 dims each
    static constexpr int kBufs = D == 256 ? 1 : 2;     // score buffers
    static constexpr uint32_t kColumns = 256;          // tensor memory for them (a power of two)
    static constexpr int kOffRing = kKBytes;
    static constexpr int kOffLse = kOffRing + kStages * kChunk;
    static constexpr int kOffSum = kOffLse + 8 * 2 * kCols * 4;
    static constexpr int kOffBar = kOffSum + 2 * kTileRows * 4;
    static constexpr int kSmem = kOffBar + 256 + 1024;
    static_assert(kSmem + 1024 <= 114 * 1024, "two CTAs per SM");
};

// entries past a prompt's length: prev's (or zero); kRest of a (prompt, head) per CTA
constexpr int kRestEach = 8, kRest = kWThreads * kRestEach;
__device__ void weights_rest(const PromptParams &p, int64_t block) {
    const int64_t per = (p.width + kRest - 1) / kRest, sh = block / per;
    if (sh >= (int64_t)p.n_seq * p.Hk) return;
    const int s = (int)(sh / p.Hk), len = cu_end(p, s) - cu_begin(p, s);
    const int64_t from = (block - sh * per) * kRest + threadIdx.x, row = sh * p.width;
    float v[kRestEach];
#pragma unroll
    for (int u = 0; u < kRestEach; ++u) {
        const int64_t i = from + kWThreads * u;
        v[u] = p.prev && i >= len && i < p.width ? p.prev[row + i] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kRestEach; ++u) {
        const int64_t i = from + kWThreads * u;
        if (i >= len && i < p.width) p.w[row + i] = v[u];
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kWThreads, 2)
    prompt_weights_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ CUtensorMap mq,
                          const __grid_constant__ CUtensorMap mk) {
    using S = WeightShape<D>;
    constexpr int BQ = S::BQ, NST = S::kStages, kCols = S::kCols;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    if ((int)blockIdx.x >= p.main_ctas) return weights_rest(p, (int)blockIdx.x - p.main_ctas);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t bars = smem_u32(smem + S::kOffBar);
    auto b_full = [&](int s) { return bars + 8u * s; };
    auto b_empty = [&](int s) { return bars + 8u * (8 + s); };
    const uint32_t b_k = bars + 8u * 16, b_final = bars + 8u * 17;
    auto b_s = [&](int buf) { return bars + 8u * (18 + buf); };     // scores in tensor memory
    auto b_read = [&](int buf) { return bars + 8u * (20 + buf); };  // scores read
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::kOffBar + 8 * 22);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + S::kOffBar + 8 * 23);
    int *place = reinterpret_cast<int *>(smem + S::kOffBar + 8 * 24);
    float *fin = reinterpret_cast<float *>(smem + S::kOffSum);  // sums by [warpgroup][key] at the end
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), ranks = (int)cl.num_blocks();
    const int block = blockIdx.x / ranks;

    const int G = p.G, TQ = BQ / G;
    const int head = block % p.Hk;
    if (warp == 9) find_unit(p, block / p.Hk, kTileRows, place);
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(S::kColumns));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(b_full(s), 1);
            mbar_init(b_empty(s), 1);
        }
        mbar_init(b_k, 1);
        mbar_init(b_final, 1);
        for (int b = 0; b < S::kBufs; ++b) {
            mbar_init(b_s(b), 1);
            mbar_init(b_read(b), 8);
        }
        *abort = p.give_up;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // query-tile rows that no box writes (BQ not a multiple of G) stay zero: their scores are finite
    for (int x = tid; x < NST * (BQ - TQ * G) * 8; x += kWThreads) {
        const int c = x & 7, r = (x >> 3) % (BQ - TQ * G), a = (x >> 3) / (BQ - TQ * G);
        *reinterpret_cast<uint4 *>(smem + S::kOffRing + a * S::kChunk + (TQ * G + r) * 128 + c * 16) = make_uint4(0, 0, 0, 0);
    }
    proxy_fence();
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = *tmem_slot;
    if (place[0] < 0) {  // the whole cluster
        if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kColumns));
        return;
    }
    const int seq = place[0], begin = place[2], L = place[3] - begin;
    const int k0 = (place[4] - 1 - place[1]) * kTileRows;  // the first keys are seen by the most rows
    int start = p.last_rows > 0 && L > p.last_rows ? L - p.last_rows : 0;  // first query token counted
    if (start < k0) start = k0;
    const int all = (L - start + TQ - 1) / TQ, ntile = (all - rank + ranks - 1) / ranks;  // this CTA: tiles rank, rank + ranks, ...
    const int64_t at = ((int64_t)seq * p.Hk + head) * p.width + k0 + tid;  // rank 0's threads: a key each at the end
    const bool writes = rank == 0 && tid < kTileRows && k0 + tid < L && k0 + tid < p.width;
    const float before = writes && p.prev ? p.prev[at] : 0.f;
    float mine = 0.f;  // this thread's part of its key's sum

    if (warp == 9) {
        if (lane == 0) {
            mbar_expect(b_k, (uint32_t)S::kKBytes);
            for (int c = 0; c < S::kChunks; ++c)
                tma_load(smem_u32(smem + c * kTileRows * 128), &mk, b_k, c * 64, head, begin + k0);
            int issued = 0;
            for (int r = 0; r < ntile * S::kChunks; ++r) {
                const int st = r % NST, use = r / NST;
                if (use > 0 && !mbar_wait(b_empty(st), (uint32_t)((use - 1) & 1), abort)) break;
                mbar_expect(b_full(st), (uint32_t)(128 * G * TQ));
                tma_load(smem_u32(smem + S::kOffRing + st * S::kChunk), &mq, b_full(st), r % S::kChunks * 64, head * G,
                         begin + start + (rank + r / S::kChunks * ranks) * TQ);
                issued = r + 1;
            }
            place[5] = issued;
        }
    } else if (warp == 8) {
        constexpr uint32_t id = idesc(BF16, kTileRows, BQ, false);
        constexpr int kPer = S::kChunks / S::kParts;
        const bool one = elect_one();
        const uint64_t da = smem_desc(smem_u32(smem), 16), dq = smem_desc(smem_u32(smem + S::kOffRing), 16);
        bool ok = !p.give_up && mbar_wait_warp(b_k, 0, abort);
        for (int r = 0; r < ntile && ok; ++r) {
            const int buf = r % S::kBufs;
#pragma unroll
            for (int c0 = 0; c0 < S::kChunks; c0 += S::kStep) {
                ok = ok && wait_warp(abort, [&] {
                    bool all = true;
#pragma unroll
                    for (int c = c0; c < c0 + S::kStep; ++c) {
                        const int x = r * S::kChunks + c;
                        all &= mbar_done(b_full(x % NST), (uint32_t)((x / NST) & 1));
                    }
                    if (c0 == 0 && r >= S::kBufs) all &= mbar_done(b_read(buf), (uint32_t)((r / S::kBufs - 1) & 1));
                    return all;
                });
                if (!ok) break;
                tc_after();
                if (one) {
#pragma unroll
                    for (int c = c0; c < c0 + S::kStep; ++c) {
                        const int st = (r * S::kChunks + c) % NST;
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            mma_ss(tmem + (uint32_t)((buf * S::kParts + c / kPer) * BQ), da + (uint64_t)((c * (kTileRows * 128) + s * 32) >> 4),
                                   dq + (uint64_t)((st * S::kChunk + s * 32) >> 4), id, c % kPer > 0 || s > 0);
                        mma_commit(b_empty(st));
                    }
                    if (c0 + S::kStep == S::kChunks) mma_commit(b_s(buf));
                }
            }
        }
        if (one) mma_commit(b_final);
    } else {
        const int half = warp >> 2, key = k0 + (tid & 127);
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const float sc = p.scale_log2;
        // every warp keeps its own copy of its columns' -lse, so that the warps run apart; the next tile's are on their
        // way from memory meanwhile
        constexpr int kRows = (kCols + 31) / 32;
        float *sl = reinterpret_cast<float *>(smem + S::kOffLse) + warp * 2 * kCols;
        const int Hq = p.Hk * G;
        int t_of[kRows];                // token of the tile that this thread's x-th row belongs to (TQ: none)
        const float *src[kRows];        // its lse in the current tile
        float next[kRows];
#pragma unroll
        for (int x = 0; x < kRows; ++x) {
            const int q = half * kCols + 32 * x + lane;
            t_of[x] = 32 * x + lane < kCols && q < TQ * G ? q / G : TQ;
            src[x] = p.lse_in + (int64_t)(begin + start + rank * TQ + q / G) * Hq + head * G + q % G;
            next[x] = t_of[x] < TQ && start + rank * TQ + t_of[x] < L ? *src[x] : INFINITY;
        }
        // Two levels: a tile's terms, then the tiles.  (In one chain, thousands of terms of a long prompt's first keys lost
        // up to 1e-4 of their sum.)
        float2 total = make_float2(0.f, 0.f);
        bool ok = true;
        for (int r = 0; r < ntile; ++r) {
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            const int buf = r % S::kBufs, tok0 = start + (rank + r * ranks) * TQ;
            float *z = sl + (r & 1) * kCols;
#pragma unroll
            for (int x = 0; x < kRows; ++x) {
                // -lse (log2 units); rows that count for nothing: -inf
                if (kCols % 32 == 0 || 32 * x + lane < kCols) z[32 * x + lane] = next[x] == -INFINITY ? -INFINITY : next[x] * -1.4426950408889634f;
                src[x] += (int64_t)ranks * TQ * Hq;
                next[x] = t_of[x] < TQ && r + 1 < ntile && tok0 + ranks * TQ + t_of[x] < L ? *src[x] : INFINITY;
            }
            __syncwarp();
            ok = mbar_wait_warp(b_s(buf), (uint32_t)((r / S::kBufs) & 1), abort);
            if (!ok) break;
            tc_after();
            // columns this key counts: rows of tokens from the key on, and none past the prompt
            const bool edge = tok0 < k0 + kTileRows - 1 || tok0 + TQ > L;
            const int c_lo = (key - tok0) * G - half * kCols;
            const int c_hi = ((L - tok0) * G < TQ * G ? (L - tok0) * G : TQ * G) - half * kCols;
            const uint32_t ts = lanes + (uint32_t)(buf * S::kParts * BQ + half * kCols);
            const float2 sc2 = make_float2(sc, sc);
            uint32_t sr[2][16];  // 16 columns at a time: the next on their way, or both parts
            auto fetch = [&](int c0) {
                tmem_ld16(ts + c0, sr[S::kParts == 2 ? 0 : c0 / 16 & 1]);
                if (S::kParts == 2) tmem_ld16(ts + BQ + c0, sr[1]);
            };
            auto scores = [&](int c0, float *s) {  // those of 16 columns, with the next ones (or the buffer's release) on their way
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 16; c += 2) {
                    const uint32_t *a = &sr[S::kParts == 2 ? 0 : c0 / 16 & 1][c];
                    float2 v = make_float2(__uint_as_float(a[0]), __uint_as_float(a[1]));
                    if (S::kParts == 2) v = add2(v, make_float2(__uint_as_float(sr[1][c]), __uint_as_float(sr[1][c + 1])));
                    s[c] = v.x, s[c + 1] = v.y;
                }
                if (c0 + 16 < kCols) {
                    fetch(c0 + 16);
                } else {
                    tc_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_read(buf));
                }
            };
            fetch(0);
            if (!edge) {
#pragma unroll
                for (int c0 = 0; c0 < kCols; c0 += 16) {
                    float s[16];
                    float4 zc[4];  // (read before the wait for the scores where the registers allow)
                    auto read = [&] {
#pragma unroll
                        for (int c = 0; c < 4; ++c) zc[c] = reinterpret_cast<const float4 *>(z + c0)[c];
                    };
                    if (S::kParts == 1) read();
                    scores(c0, s);
                    if (S::kParts == 2) read();
#pragma unroll
                    for (int c = 0; c < 16; c += 4) {
                        const float2 a = fma2(make_float2(s[c], s[c + 1]), sc2, make_float2(zc[c / 4].x, zc[c / 4].y));
                        const float2 b = fma2(make_float2(s[c + 2], s[c + 3]), sc2, make_float2(zc[c / 4].z, zc[c / 4].w));
                        sum[0] = add2(sum[0], make_float2(ex2(a.x), ex2(a.y)));
                        sum[1] = add2(sum[1], make_float2(ex2(b.x), ex2(b.y)));
                    }
                }
            } else {
#pragma unroll
                for (int c0 = 0; c0 < kCols; c0 += 16) {
                    float s[16];
                    scores(c0, s);
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float e = ex2(fmaf(s[c], sc, z[c0 + c]));
                        sum[c & 1].x += c0 + c >= c_lo && c0 + c < c_hi ? e : 0.f;
                    }
                }
            }
            total = add2(total, add2(sum[0], sum[1]));
        }
        mine = ok ? total.x + total.y : __int_as_float(0x7fc00000);
    }
    // every MMA is done, every score read: the sums of a key meet in shared memory, then over the cluster
    if (tid == 0) mbar_drain(b_final, 0);
    tc_before();
    __syncthreads();
    tc_after();
    if (tid == 9 * 32 && *abort) {  // copies that no one waited for (as in the attention)
        const int issued = place[5];
        mbar_drain(b_k, 0);
        for (int st = 0; st < NST; ++st)
            if (issued > st) mbar_drain(b_full(st), (uint32_t)(((issued - 1 - st) / NST) & 1));
    }
    if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kColumns));
    if (warp < 8) fin[tid] = mine;
    if (ranks > 1) cl.sync();
    else __syncthreads();
    if (writes) {
        float total = 0.f;
        for (int r = 0; r < ranks; ++r) {
            const float *f = cl.map_shared_rank(fin, r);
            total += f[tid] + f[kTileRows + tid];
        }
        p.w[at] = before + total;
    }
    if (ranks > 1) cl.sync();  // no CTA leaves while another may read its sums
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

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {  // the driver's entry point, looked up once
    static std::once_flag once;
    static EncodeFn fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) == cudaSuccess &&
            r == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(p);
    });
    return fn;
}

// [rows][heads][D] of 16-bit elements as boxes of 64 elements x box_heads x box_rows, 128-byte swizzle
kvs_status make_map(CUtensorMap *m, const void *base, bool bf16, uint64_t rows, uint64_t heads, uint64_t D, uint64_t stride,
                    uint32_t box_heads, uint32_t box_rows) {
    EncodeFn fn = encoder();
    if (!fn) return bad(KVS_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const cuuint64_t dims[3] = {D, heads, rows}, strides[2] = {D * 2, stride * 2};
    const cuuint32_t box[3] = {64, box_heads, box_rows}, es[3] = {1, 1, 1};
    const CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(base),
                          dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return bad(KVS_ERR_CUDA, "cuTensorMapEncodeTiled refused a row layout");
    return KVS_OK;
}

kvs_status check_prompt(const kvs_prompt *p, bool need_v, PromptParams *o) {
    if (!p) return bad(KVS_ERR_INVALID, "null prompt");
    if (!(p->head_dim == 64 || p->head_dim == 128 || p->head_dim == 256)) return bad(KVS_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
    if (p->dtype != KVS_F16 && p->dtype != KVS_BF16) {
        if (p->dtype == KVS_F32) return bad(KVS_ERR_UNSUPPORTED, "prompts are KVS_F16 or KVS_BF16");
        return bad(KVS_ERR_INVALID, "dtype must be KVS_F16 or KVS_BF16");
    }
    if (p->n_kv_head == 0 || p->n_q_head < p->n_kv_head || p->n_q_head % p->n_kv_head != 0 || p->n_q_head > 65535)
        return bad(KVS_ERR_INVALID, "n_q_head must be a positive multiple of n_kv_head, at most 65535");
    if (p->n_q_head / p->n_kv_head > (uint32_t)kMaxGroup) return bad(KVS_ERR_UNSUPPORTED, "n_q_head / n_kv_head must be at most 64");
    if (p->n_seq > (uint32_t)kMaxSeq) return bad(KVS_ERR_UNSUPPORTED, "n_seq must be at most 4096");
    if (p->total_rows > 0x7fffffffu - 256u) return bad(KVS_ERR_INVALID, "total_rows must be at most 2^31 - 1 - 256");
    if (!(p->scale > 0.f) || !isfinite(p->scale)) return bad(KVS_ERR_INVALID, "scale must be positive and finite");
    if (!p->cu) return bad(KVS_ERR_INVALID, "null cu");
    if (p->total_rows) {
        const uint64_t q_row = (uint64_t)p->n_q_head * p->head_dim, k_row = (uint64_t)p->n_kv_head * p->head_dim;
        if (!p->q || !p->k || (need_v && !p->v)) return bad(KVS_ERR_INVALID, "null q, k or v");
        if (!aligned(p->q, 16) || !aligned(p->k, 16) || (need_v && !aligned(p->v, 16)) || p->q_stride % 8 || p->k_stride % 8 ||
            (need_v && p->v_stride % 8) || p->q_stride < q_row || p->k_stride < k_row || (need_v && p->v_stride < k_row))
            return bad(KVS_ERR_INVALID, "rows must start on 16-byte boundaries, at least heads * head_dim apart");
        const uint64_t most = 1ull << 38;  // bytes between rows that a tensor map holds (below 2^40)
        if (p->q_stride > most || p->k_stride > most || (need_v && p->v_stride > most)) return bad(KVS_ERR_INVALID, "row stride too large");
    }
    o->cu = p->cu;
    o->n_seq = (int)p->n_seq;
    o->total = (int)p->total_rows;
    o->Hk = (int)p->n_kv_head;
    o->G = (int)(p->n_q_head / p->n_kv_head);
    o->scale_log2 = p->scale * 1.4426950408889634f;
    return KVS_OK;
}

template <typename... A>
cudaError_t launch(void (*kernel)(A...), dim3 grid, int smem, cudaStream_t s, const A &...a) {
    const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(kernel), smem);
    if (e != cudaSuccess) return e;
    void *args[] = {const_cast<void *>(static_cast<const void *>(&a))...};
    return cudaLaunchKernel(reinterpret_cast<const void *>(kernel), grid, dim3(kThreads), args, smem, s);
}

template <int D, bool WIN>
kvs_status attend_for(const kvs_prompt *p, PromptParams pp, cudaStream_t s) {
    using S = AttendShape<D>;
    const bool bf = p->dtype == KVS_BF16;
    const uint32_t TQ = kTileRows / pp.G;
    CUtensorMap mq, mk, mv;
    kvs_status r = make_map(&mq, p->q, bf, p->total_rows, p->n_q_head, D, p->q_stride, (uint32_t)pp.G, TQ);
    if (r == KVS_OK) r = make_map(&mk, p->k, bf, p->total_rows, p->n_kv_head, D, p->k_stride, 1, S::BN);
    if (r == KVS_OK) r = make_map(&mv, p->v, bf, p->total_rows, p->n_kv_head, D, p->v_stride, 1, S::kVKeys);
    if (r != KVS_OK) return r;
    const uint64_t units = (uint64_t)p->total_rows / (S::NQ * TQ) + p->n_seq;  // at least the prompts' tile groups
    if (units * p->n_kv_head > 0x7fffffffull) return bad(KVS_ERR_UNSUPPORTED, "too many tiles for one launch");
    unsigned ctas = (unsigned)(units * p->n_kv_head);
    if (WIN) {
        pp.units = (int)ctas;
        const unsigned sms = (unsigned)current_device_sms();
        ctas = ctas < sms ? ctas : sms;
    }
    const cudaError_t e = launch(bf ? prompt_attend_kernel<D, true, WIN> : prompt_attend_kernel<D, false, WIN>, dim3(ctas), S::kSmem, s,
                                 pp, mq, mk, mv);
    return e == cudaSuccess ? KVS_OK : cuda_failed("prompt attention launch", e);
}

// How many CTAs share a key tile's rows.  A CTA costs kStart tiles before and after its own; a unit's tiles go from none
// to the prompt's over all rows (half of them on average; the longest of several prompts is taken for 1.5 times the
// mean, which is all the host knows), or are the window's.  The launch ends no sooner than its whole cost spread over the
// slots, and than its longest CTA: the least of that over 1, 2, 4 and 8.  Measured on 5 batches, in us for 1 / 2 / 4 / 8:
// 33 units of 256 tiles 220 / 114 / 61 / 38, 64 of 8 13 / 11 / 9.5 / 15, 154 of 196 432 / 224 / 134 / 143, 488 of 57
// 140 / 122 / 139 / 179, 616 of 18 41 / 50 / 72 / 114.
unsigned sharing_ctas(uint64_t units, uint64_t slots, uint64_t tiles, bool several, uint64_t window) {
    constexpr double kStart = 8;
    const bool windowed = window > 0 && window < tiles;
    const double all = (double)(windowed ? window : tiles), mean = windowed ? all : all / 2;
    const double longest = windowed || !several ? all : 1.5 * all;
    unsigned best = 1;
    double least = 0;
    for (unsigned r = 1; r <= 8; r *= 2) {
        const double spread = (double)units * (r * kStart + mean) / (double)slots, end = kStart + longest / r;
        const double cost = spread > end ? spread : end;
        if (r == 1 || cost < least) best = r, least = cost;
    }
    return best;
}

template <int D>
kvs_status weights_for(const kvs_prompt *p, PromptParams pp, cudaStream_t s) {
    using S = WeightShape<D>;
    const bool bf = p->dtype == KVS_BF16;
    CUtensorMap mq = {}, mk = {};
    uint64_t ctas = 0;
    unsigned ranks = 1;
    if (p->total_rows) {
        kvs_status r = make_map(&mq, p->q, bf, p->total_rows, p->n_q_head, D, p->q_stride, (uint32_t)pp.G, (uint32_t)(S::BQ / pp.G));
        if (r == KVS_OK) r = make_map(&mk, p->k, bf, p->total_rows, p->n_kv_head, D, p->k_stride, 1, kTileRows);
        if (r != KVS_OK) return r;
        ctas = ((uint64_t)p->total_rows / kTileRows + p->n_seq) * p->n_kv_head;
        ranks = sharing_ctas(ctas, 2 * (uint64_t)current_device_sms(), (uint64_t)p->total_rows * pp.G / S::BQ / p->n_seq, p->n_seq > 1,
                             (uint64_t)pp.last_rows * pp.G / S::BQ);
    }
    const uint64_t rest = pp.prev != pp.w ? (uint64_t)p->n_seq * p->n_kv_head * (((uint64_t)pp.width + kRest - 1) / kRest) : 0;
    const uint64_t grid = (ctas * ranks + rest + ranks - 1) / ranks * ranks;
    if (grid > 0x7fffffffull) return bad(KVS_ERR_UNSUPPORTED, "total_rows or n_seq * n_kv_head * width too large for one launch");
    if (grid == 0) return KVS_OK;
    pp.main_ctas = (int)(ctas * ranks);
    auto kernel = bf ? prompt_weights_kernel<D, true> : prompt_weights_kernel<D, false>;
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(kernel), S::kSmem);
    if (e != cudaSuccess) return cuda_failed("prompt weights launch", e);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kWThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, pp, mq, mk);
    return e == cudaSuccess ? KVS_OK : cuda_failed("prompt weights launch", e);
}

}  // namespace
}  // namespace kvs

using namespace kvs;

template <bool WIN>
static kvs_status attend_call(const kvs_prompt *p, uint32_t window, uint32_t sinks, void *out, uint64_t out_stride, float *lse, void *stream) {
    PromptParams pp = {};
    const kvs_status s = check_prompt(p, true, &pp);
    if (s != KVS_OK) return s;
    if (p->total_rows && (!out || !aligned(out, 16) || out_stride % 8 || out_stride < (uint64_t)p->n_q_head * p->head_dim))
        return bad(KVS_ERR_INVALID, "out rows must start on 16-byte boundaries, at least n_q_head * head_dim apart");
    if (p->total_rows == 0 || p->n_seq == 0) return KVS_OK;
    const uint32_t fault = batch_fault();
    pp.give_up = fault == KVS_FAULT_DEVICE_WAIT;
    pp.late = fault == KVS_FAULT_DEVICE_LATE;
    pp.out = out;
    pp.out_stride = (int64_t)out_stride;
    pp.lse = lse;
    pp.window = (int)window;
    pp.sinks = (int)sinks;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return p->head_dim == 64    ? attend_for<64, WIN>(p, pp, st)
           : p->head_dim == 128 ? attend_for<128, WIN>(p, pp, st)
                                : attend_for<256, WIN>(p, pp, st);
}

extern "C" kvs_status kvs_prompt_attend(const kvs_prompt *p, void *out, uint64_t out_stride, float *lse, void *stream) {
    return attend_call<false>(p, 0, 0, out, out_stride, lse, stream);
}

extern "C" kvs_status kvs_prompt_attend_window(const kvs_prompt *p, uint32_t window, uint32_t sinks, void *out, uint64_t out_stride,
                                               float *lse, void *stream) {
    if (!p) return bad(KVS_ERR_INVALID, "null prompt");
    if (window > 0x7fffffffu || sinks > 0x7fffffffu - 64u) return bad(KVS_ERR_INVALID, "window must be at most 2^31 - 1, sinks 2^31 - 65");
    if (window == 0 || window >= p->total_rows) return attend_call<false>(p, 0, 0, out, out_stride, lse, stream);  // every key is inside
    // (sinks past the rows stand for all of them)
    return attend_call<true>(p, window, sinks < p->total_rows ? sinks : p->total_rows, out, out_stride, lse, stream);
}

extern "C" kvs_status kvs_prompt_weights(const kvs_prompt *p, const float *lse, uint32_t last_rows, const float *prev,
                                         float *weights, uint64_t width, void *stream) {
    PromptParams pp = {};
    kvs_status s = check_prompt(p, false, &pp);
    if (s != KVS_OK) return s;
    if (p->n_seq && width && ((p->total_rows && !lse) || !weights)) return bad(KVS_ERR_INVALID, "null lse or weights");
    if (width > 0x7fffffffull) return bad(KVS_ERR_INVALID, "width must be at most 2^31 - 1");
    if (p->n_seq == 0 || width == 0) return KVS_OK;
    pp.give_up = batch_fault() == KVS_FAULT_DEVICE_WAIT;
    pp.lse_in = lse;
    pp.prev = prev;
    pp.w = weights;
    pp.width = (int64_t)width;
    pp.last_rows = last_rows > 0x7fffffffu ? 0x7fffffff : (int)last_rows;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return p->head_dim == 64 ? weights_for<64>(p, pp, st) : p->head_dim == 128 ? weights_for<128>(p, pp, st) : weights_for<256>(p, pp, st);
}
