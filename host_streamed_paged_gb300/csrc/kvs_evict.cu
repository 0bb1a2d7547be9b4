// Eviction from the 4-bit page cache by accumulated attention weight
// (include/kvs.h, kvs_q4_evict): per (sequence, kv head) a selection of the
// tokens that stay, then a gather of their encoded rows into other pages.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include <string>
#include <type_traits>

#include "kvs.h"
#include "kvs_internal.h"

namespace kvs {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kShare = 49152;  // keys of a CTA that fit its shared memory (192 KB)
constexpr int kMaxSeq = 4096;
constexpr int kBins = 256;
constexpr int kCopies = 16;

struct EvictParams {
    uint8_t *pages;
    int64_t n_pages, page_bytes, head_bytes;
    int P, lgP, Hk;
    const int32_t *table, *dst_table, *lens;
    int table_width, dst_width, n_seq;
    const float *weights;
    int64_t width;
    int keep, sinks, recent;
    int32_t *kept;
    float *kept_weights;
    int32_t *new_lens;
};

__device__ __forceinline__ int seq_len(const EvictParams &p, int s) {
    int64_t cap = (int64_t)p.table_width << p.lgP;
    if (p.width < cap) cap = p.width;
    const int n = p.lens[s];
    return n < 0 ? 0 : (int)(n < cap ? n : cap);
}

// fp32 order as unsigned order; -0 equals 0, NaN is below every number
__device__ __forceinline__ uint32_t key_of(float x) {
    if (isnan(x)) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}

// One cluster per (sequence, kv head); each CTA has a contiguous share of the
// candidates (tokens between the sinks and the recent ones), each of its warps
// a contiguous part of that, their keys in shared memory.  (In registers, 16 a
// thread, they leave an SM one CTA of 1024 threads, which took 1.6 times as
// long on the batch below.)  The smallest key that stays is found digit by
// digit, 8 bits at a time from the top: a histogram of the candidates that
// match the digits so far, summed over the cluster, gives the next digit.  Then
// every warp, from the counts of those before it, writes its tokens in order:
// keys above the threshold, and of those equal to it the first ones.
// KEPT = false is for shares beyond kShare keys: they are read again each time.
// What bounds it is the longest sequence's chain of loads, passes and cluster
// barriers: 36 us on 8 sequences of 131072 to 700 tokens, 8 heads, of which
// 4096 stay.  The host sizes the keys' memory by what a table can hold (it does
// not know the lengths), 64 KB a CTA there beside 21 KB of counts: two CTAs fit
// an SM, and the 512 of that batch begin in two waves.
template <bool KEPT>
__global__ void __launch_bounds__(kThreads) select_kernel(const EvictParams p) {
    extern __shared__ uint32_t keys[];
    constexpr int kW = kThreads / 32;
    __shared__ uint32_t hist[kCopies][kBins + 1];  // a digit's counts; lanes of a warp count in different copies, since
                                                   // most weights share a few top digits
    __shared__ uint32_t sums[2][kBins];  // of the copies, read by the whole cluster; two, for digits in turn
    __shared__ uint32_t part[2][kBins];  // the cluster's counts, by four CTAs each
    __shared__ uint32_t count[2][kW];    // a warp's tokens above the threshold, and equal to it
    __shared__ uint32_t mine[2];         // this CTA's tokens above the threshold, and equal to it
    __shared__ uint32_t digit[2];
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cl.block_rank(), ranks = (int)cl.num_blocks();
    const int id = blockIdx.x / ranks, s = id / p.Hk, h = id % p.Hk;
    const int T = seq_len(p, s);
    int32_t *kept = p.kept + (int64_t)id * p.keep;
    float *kw = p.kept_weights ? p.kept_weights + (int64_t)id * p.keep : nullptr;
    const float *w = p.weights + (int64_t)id * p.width;
    if (h == 0 && rank == 0 && tid == 0) p.new_lens[s] = T < p.keep ? T : p.keep;
    if (T <= p.keep) {  // all stay (the same decision in every CTA of the cluster)
        for (int i = rank * kThreads + tid; i < p.keep; i += ranks * kThreads) {
            kept[i] = i < T ? i : -1;
            if (kw) kw[i] = i < T ? w[i] : 0.f;
        }
        return;
    }
    const int n = T - p.sinks - p.recent;          // candidates
    const int want = p.keep - p.sinks - p.recent;  // of which these stay
    const int share = (n + ranks - 1) / ranks;
    const int c0 = min(rank * share, n), c1 = min(c0 + share, n), cn = c1 - c0;
    const float *wc = w + p.sinks + c0;
    const int part_n = (share + 32 * kW - 1) / (32 * kW) * 32;  // this warp's candidates: i = at, at + 32, ... below end
    const int at = min(warp * part_n, cn) + lane, end = min((warp + 1) * part_n, cn);
    if (KEPT) {
#pragma unroll 16
        for (int i = at; i < end; i += 32) keys[i] = key_of(wc[i]);
    }
    auto key_at = [&](int i) { return KEPT ? keys[i] : key_of(wc[i]); };
    for (int i = tid; i < kCopies * (kBins + 1); i += kThreads) (&hist[0][0])[i] = 0;
    __syncthreads();
    uint32_t *mine_h = hist[lane & (kCopies - 1)];
    uint32_t prefix = 0;
    uint32_t left = (uint32_t)want;  // still to be found among the keys that match the prefix
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
#pragma unroll 8
        for (int i = at; i < end; i += 32) {
            const uint32_t k = key_at(i);
            if (pass == 0 || (k >> (shift + 8)) == prefix) atomicAdd(&mine_h[k >> shift & 255], 1u);
        }
        __syncthreads();
        uint32_t *own = sums[pass & 1];
        if (tid < kBins) {
            uint32_t sum = 0;
#pragma unroll
            for (int c = 0; c < kCopies; ++c) {
                sum += hist[c][tid];
                hist[c][tid] = 0;
            }
            own[tid] = sum;
        }
        cl.sync();
        {
            const int r0 = tid >> 8 << 2, bin = tid & 255;
            uint32_t v[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = r0 + r < ranks ? *cl.map_shared_rank(&own[bin], r0 + r) : 0u;
            part[tid >> 8][bin] = v[0] + v[1] + v[2] + v[3];
        }
        __syncthreads();
        if (warp == 0) {  // from the top: the digit at which the count reaches `left`
            uint32_t v[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int bin = 255 - (lane * 8 + i);
                sum += v[i] = part[0][bin] + part[1][bin];
            }
            uint32_t inc = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += x;
            }
            uint32_t before = inc - sum;
            if (before < left && inc >= left) {
                int i = 0;
                for (; i < 7 && before + v[i] < left; ++i) before += v[i];
                digit[0] = 255 - (lane * 8 + i);
                digit[1] = before;
            }
        }
        __syncthreads();
        if (want > 0) {
            prefix = prefix << 8 | digit[0];
            left -= digit[1];
        }
    }
    // prefix is the threshold key; `left` tokens equal to it stay
    if (want == 0) prefix = 0xffffffffu, left = 0;
    uint32_t mine_a = 0, mine_e = 0;
#pragma unroll 8
    for (int i = at; i < end; i += 32) {
        const uint32_t k = key_at(i);
        mine_a += k > prefix;
        mine_e += k == prefix;
    }
    mine_a = __reduce_add_sync(0xffffffffu, mine_a);
    mine_e = __reduce_add_sync(0xffffffffu, mine_e);
    if (lane == 0) count[0][warp] = mine_a, count[1][warp] = mine_e;
    __syncthreads();
    if (tid < 2) {
        uint32_t sum = 0;
        for (int x = 0; x < kW; ++x) sum += count[tid][x];
        mine[tid] = sum;
    }
    cl.sync();
    // places taken, and equals seen, before this warp's part
    uint32_t out = (uint32_t)p.sinks, equal = 0;
    if (lane < 2) {
        uint32_t sum = 0;
        for (int r = 0; r < rank; ++r) sum += cl.map_shared_rank(mine, r)[lane];
        for (int x = 0; x < warp; ++x) sum += count[lane][x];
        out += sum;
        equal = sum;
    }
    out = __shfl_sync(0xffffffffu, out, 0);
    equal = __shfl_sync(0xffffffffu, equal, 1);
    const uint32_t below = (1u << lane) - 1;
#pragma unroll 4
    for (int i0 = at - lane; i0 < end; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < end ? key_at(i) : 0u;
        const bool a = i < end && k > prefix, e = i < end && k == prefix;
        const uint32_t ba = __ballot_sync(0xffffffffu, a), be = __ballot_sync(0xffffffffu, e);
        const uint32_t ne = equal + __popc(be & below);
        if (a || (e && ne < left)) {
            const uint32_t to = out + __popc(ba & below) + min(ne, left);
            const int tok = p.sinks + c0 + i;
            kept[to] = tok;
            // the key is the weight, but for NaN and the two zeros
            if (kw) kw[to] = k == 0u || k == 0x80000000u ? w[tok] : __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k);
        }
        out += __popc(ba);
        equal += __popc(be);
    }
    // the ones that always stay
    for (int i = rank * kThreads + tid; i < p.sinks + p.recent; i += ranks * kThreads) {
        const int tok = i < p.sinks ? i : T - p.recent + (i - p.sinks);
        const int to = i < p.sinks ? i : p.keep - p.recent + (i - p.sinks);
        kept[to] = tok;
        if (kw) kw[to] = w[tok];
    }
    cl.sync();  // no CTA leaves while another may read its shared memory
}

// Gather: a warp builds one destination tile (32 tokens of one head) in shared
// memory and stores it in whole lines.  Its reads are pieces of 16 bytes; lanes
// that read one token's sit side by side, as many to a line as the layout has.
// Bound by what a token's rows take from memory: its V codes share 32-byte
// sectors with seven other tokens, so up to eight times their bytes are read.
// (The batch above, D 128, 66 MB of rows moved: 33 us, 144 MB read; 3 us more
// with a token to a lane, 900 line accesses a tile for 400.)
template <int D>
__global__ void __launch_bounds__(128) gather_kernel(const EvictParams p) {
    constexpr int NB = D / 32, BYTES = 36 * D;
    __shared__ __align__(16) uint8_t stage[4][BYTES];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tiles = (p.keep + 31) / 32;
    const int64_t id = (int64_t)blockIdx.x * 4 + warp;
    const int k = (int)(id % tiles);
    const int64_t sh = id / tiles;
    if (sh >= (int64_t)p.n_seq * p.Hk) return;
    const int s = (int)(sh / p.Hk), h = (int)(sh % p.Hk);
    const int T = seq_len(p, s), count = T < p.keep ? T : p.keep;
    if (k * 32 >= count) return;
    const int dpage = p.dst_table[(int64_t)s * p.dst_width + (k * 32 >> p.lgP)];
    if (dpage < 0 || dpage >= p.n_pages) return;
    uint8_t *dst = p.pages + dpage * p.page_bytes + h * p.head_bytes + (int64_t)((k * 32 & (p.P - 1)) >> 5) * BYTES;
    const int i = k * 32 + lane;
    const uint8_t *src = nullptr;
    int st = 0;
    if (i < count) {
        const int tok = p.kept[sh * p.keep + i];
        const int page = p.table[(int64_t)s * p.table_width + (tok >> p.lgP)];
        if (page >= 0 && page < p.n_pages)
            src = p.pages + page * p.page_bytes + h * p.head_bytes + (int64_t)((tok & (p.P - 1)) >> 5) * BYTES;
        st = tok & 31;
    }
    uint8_t *out = stage[warp];
    // scales, lane = token: K's of a token lie within NB words (the other halves are those of the token 8 on), V's within
    // NB / 2 16-byte units
    {
        const uint32_t *kw = reinterpret_cast<const uint32_t *>(src + 16 * D) + ((st >> 4) * 8 + (st & 7)) * NB;
        const uint4 *vw = reinterpret_cast<const uint4 *>(src + 34 * D) + (st >> 2) * (NB / 2);
        uint32_t ks[NB];
        uint4 vs[NB / 2];
        using Words = typename std::conditional<NB == 2, uint2, uint4>::type;
        constexpr int kWords = sizeof(Words) / 4;
#pragma unroll
        for (int b = 0; b < NB; b += kWords) {
            const Words x = src ? *reinterpret_cast<const Words *>(kw + b) : Words{};
#pragma unroll
            for (int c = 0; c < kWords; ++c) ks[b + c] = reinterpret_cast<const uint32_t *>(&x)[c];
        }
#pragma unroll
        for (int b = 0; b < NB / 2; ++b) vs[b] = src ? vw[b] : make_uint4(0, 0, 0, 0);
        uint16_t *ko = reinterpret_cast<uint16_t *>(out + 16 * D) + ((lane >> 4) * 8 + (lane & 7)) * NB * 2 + (lane >> 3 & 1);
        uint16_t *vo = reinterpret_cast<uint16_t *>(out + 34 * D) + (lane >> 2) * NB * 4 + (lane & 3);
        const int k_sh = (st >> 3 & 1) * 16, v_sh = (st & 1) * 16;
#pragma unroll
        for (int b = 0; b < NB; ++b) ko[2 * b] = (uint16_t)(ks[b] >> k_sh);
#pragma unroll
        for (int b = 0; b < NB / 2; ++b) {
            vo[8 * b] = (uint16_t)(((st & 2) ? vs[b].y : vs[b].x) >> v_sh);
            vo[8 * b + 4] = (uint16_t)(((st & 2) ? vs[b].w : vs[b].z) >> v_sh);
        }
    }
    const unsigned long long from = reinterpret_cast<unsigned long long>(src);
    auto source = [&](int token, int *row) {  // of another lane's token
        *row = __shfl_sync(0xffffffffu, st, token);
        return reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, from, token));
    };
    // K codes: 4 lanes a token, which read 4 neighbouring pieces of min(16, NB * 4) bytes per 4 blocks (D = 64: two octets
    // share a 16-byte vector)
    using Piece = typename std::conditional<NB == 2, uint2, uint4>::type;
    constexpr int kGroups = NB <= 4 ? 1 : NB / 4;
    auto k_at = [&](int tok, int grp, int q) {
        const int u = (tok >> 3) * NB + grp * 4;
        return (((u >> 2) * 32) + (tok & 7) * 4 + q) * 16 + (u & 3) * 4;
    };
    Piece kp[4][kGroups];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        int row;
        const uint8_t *at = source(8 * r + (lane >> 2), &row);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) kp[r][g] = at ? *reinterpret_cast<const Piece *>(at + k_at(row, g, lane & 3)) : Piece{};
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int g = 0; g < kGroups; ++g) *reinterpret_cast<Piece *>(out + k_at(8 * r + (lane >> 2), g, lane & 3)) = kp[r][g];
    // V codes: a 16-byte unit is 4 tokens x 2 blocks x 2 bytes, and a token's 8 units of two blocks lie 64 bytes apart: 8
    // lanes a token, 4 tokens at a time, which are those of a destination unit.  A lane has two bytes of either block; it
    // and the next token's lane exchange halves, the even one then has a word of the first block, the odd one of the second.
    auto v_at = [&](int tok, int bp, int j) { return 18 * D + ((((tok >> 4) * (NB / 2) + bp) * 32) + j * 4 + ((tok & 15) >> 2)) * 16; };
    const int j = lane & 7, odd = lane >> 3 & 1, half = lane >> 4;
    constexpr int kRounds = NB == 8 ? 2 : 4;  // rounds whose loads are in flight together
#pragma unroll
    for (int r0 = 0; r0 < 8; r0 += kRounds) {
        uint4 v[kRounds][NB / 2];
        int row[kRounds];
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const uint8_t *at = source(4 * (r0 + r) + (lane >> 3), &row[r]);
#pragma unroll
            for (int bp = 0; bp < NB / 2; ++bp)
                v[r][bp] = at ? *reinterpret_cast<const uint4 *>(at + v_at(row[r], bp, j)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
#pragma unroll
            for (int bp = 0; bp < NB / 2; ++bp) {
                const int sh = (row[r] & 1) * 16;
                const uint32_t first = ((row[r] & 2) ? v[r][bp].y : v[r][bp].x) >> sh & 0xffffu;
                const uint32_t second = ((row[r] & 2) ? v[r][bp].w : v[r][bp].z) >> sh & 0xffffu;
                const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? first : second, 8);
                *reinterpret_cast<uint32_t *>(out + v_at(4 * (r0 + r), bp, j) + 8 * odd + 4 * half) =
                    odd ? other | second << 16 : first | other << 16;
            }
        }
    }
    __syncwarp();
    for (int x = lane; x < BYTES / 16; x += 32) reinterpret_cast<uint4 *>(dst)[x] = reinterpret_cast<const uint4 *>(out)[x];
}

kvs_status bad(kvs_status s, const char *why) {
    set_thread_error(why);
    return s;
}
kvs_status cuda_failed(const char *what, cudaError_t e) {
    cudaGetLastError();  // the call's own: no later one is to find it
    set_thread_error(std::string(what) + ": " + cudaGetErrorString(e));
    return KVS_ERR_CUDA;
}

}  // namespace
}  // namespace kvs

using namespace kvs;

extern "C" kvs_status kvs_q4_evict(const kvs_q4_pool *pool, const int32_t *table, uint32_t table_width,
                                   const int32_t *dst_table, uint32_t dst_width, const int32_t *lens, uint32_t n_seq,
                                   const float *weights, uint64_t width, uint32_t keep, uint32_t sinks, uint32_t recent,
                                   int32_t *kept, float *kept_weights, int32_t *new_lens, void *stream) {
    if (!pool) return bad(KVS_ERR_INVALID, "null pool");
    const uint32_t P = pool->page_tokens, D = pool->head_dim;
    if (!(P == 32 || P == 64 || P == 128 || P == 256) || !(D == 64 || D == 128 || D == 256))
        return bad(KVS_ERR_UNSUPPORTED, "page_tokens must be 32..256 (power of two), head_dim 64, 128 or 256");
    if (pool->n_kv_head == 0 || pool->n_kv_head > 65535) return bad(KVS_ERR_INVALID, "n_kv_head must be 1 .. 65535");
    if (!pool->pages || (reinterpret_cast<uintptr_t>(pool->pages) & 15)) return bad(KVS_ERR_INVALID, "pages null or not 16-byte aligned");
    if (pool->n_pages == 0 || pool->n_pages > 0x7fffffffull) return bad(KVS_ERR_INVALID, "n_pages must be 1 .. 2^31 - 1");
    if (n_seq > (uint32_t)kMaxSeq) return bad(KVS_ERR_UNSUPPORTED, "n_seq must be at most 4096");
    if (n_seq && (!table || !dst_table || !lens || !weights || !kept || !new_lens)) return bad(KVS_ERR_INVALID, "null table, dst_table, lens, weights, kept or new_lens");
    if (table_width < 1 || (uint64_t)table_width * P > 0x7fffffc0ull) return bad(KVS_ERR_INVALID, "table_width * page_tokens must be 1 .. 2^31 - 64");
    if (width < 1 || width > 0x7fffffffull) return bad(KVS_ERR_INVALID, "width must be 1 .. 2^31 - 1");
    if (keep < 1 || (uint64_t)sinks + recent > keep) return bad(KVS_ERR_INVALID, "need keep >= 1 and sinks + recent <= keep");
    if (keep > 0x7fffffc0u || (uint64_t)dst_width * P < keep) return bad(KVS_ERR_CAPACITY, "dst_width * page_tokens must reach keep");
    if (n_seq && kept_weights == weights) return bad(KVS_ERR_INVALID, "kept_weights must not be weights");
    if (n_seq && new_lens == lens) return bad(KVS_ERR_INVALID, "new_lens must not be lens");
    if (n_seq == 0) return KVS_OK;
    EvictParams p = {};
    p.pages = static_cast<uint8_t *>(pool->pages);
    p.n_pages = (int64_t)pool->n_pages;
    p.P = (int)P;
    p.lgP = P == 32 ? 5 : P == 64 ? 6 : P == 128 ? 7 : 8;
    p.Hk = (int)pool->n_kv_head;
    p.head_bytes = (int64_t)P * D * 9 / 8;
    p.page_bytes = p.head_bytes * p.Hk;
    p.table = table;
    p.dst_table = dst_table;
    p.lens = lens;
    p.table_width = (int)table_width;
    p.dst_width = (int)(dst_width > 0x7fffffffu ? 0x7fffffffu : dst_width);
    p.n_seq = (int)n_seq;
    p.weights = weights;
    p.width = (int64_t)width;
    p.keep = (int)keep;
    p.sinks = (int)sinks;
    p.recent = (int)recent;
    p.kept = kept;
    p.kept_weights = kept_weights;
    p.new_lens = new_lens;
    const uint64_t sh = (uint64_t)n_seq * pool->n_kv_head;
    // Up to 4096 keys one CTA is enough; beyond, a cluster of up to the 8 CTAs that every launch may have.
    uint64_t most = (uint64_t)table_width * P;
    if (width < most) most = width;
    int ranks = 1;
    while (ranks < 8 && (uint64_t)ranks * 4096 < most) ranks *= 2;
    if (sh * ranks > 0x7fffffffull) return bad(KVS_ERR_UNSUPPORTED, "n_seq * n_kv_head too large");
    const uint64_t tiles = sh * ((keep + 31) / 32);
    if ((tiles + 3) / 4 > 0x7fffffffull) return bad(KVS_ERR_UNSUPPORTED, "n_seq * n_kv_head * keep too large");
    const uint64_t share = (most + ranks - 1) / ranks;
    const bool kept_keys = share <= (uint64_t)kShare;
    auto select = kept_keys ? select_kernel<true> : select_kernel<false>;
    const int smem = kept_keys ? (int)(share * 4 + 15) / 16 * 16 : 0;
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(select), smem);
    if (e != cudaSuccess) return cuda_failed("evict launch", e);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sh * ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, select, p);
    if (e != cudaSuccess) return cuda_failed("evict launch", e);
    void (*g)(EvictParams) = D == 64 ? gather_kernel<64> : D == 128 ? gather_kernel<128> : gather_kernel<256>;
    void *args[] = {&p};
    e = cudaLaunchKernel(reinterpret_cast<const void *>(g), dim3((unsigned)((tiles + 3) / 4)), dim3(128), args, 0, st);
    return e == cudaSuccess ? KVS_OK : cuda_failed("evict launch", e);
}
