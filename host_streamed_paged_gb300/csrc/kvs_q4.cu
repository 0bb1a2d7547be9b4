// The 4-bit page cache of the batch operators (include/kvs.h): Q4_0 rows in,
// values out, attention over the pages, accumulated attention weight.
//
// Attention over a cache is bound by the bytes of the cache: 9/16 byte per
// element, each used by the few query rows of its sequence only.  At the card's
// copy rate an SM gets 23 bytes per clock, 40 cached elements, so what counts
// beside the copies is the instructions spent per element.  The layout and the
// arithmetic keep those low:
//  - A nibble ANDed out of a word and read as f16 is the subnormal n * 2^-24
//    (or 16 n * 2^-24 for the high nibble of a byte), exactly.  It goes into
//    the tensor core like that: one AND per two elements, no conversion.  The
//    factors are powers of two, taken back from the query (high-nibble dims
//    / 16) and once from the result.
//  - The codes' offset 8 leaves the sum: sum q (n - 8) = sum q n - 8 sum q.
//    For scores -8 sum q is the accumulator's initial value per block; for
//    outputs -8 sum p is one more MMA per block, over the same rounded p.
//  - The tensor core cuts a product off some 24 bits below the largest
//    exponent of its sum, and takes a subnormal's for 2^-14: codes like that
//    leave 17 bits, enough beside f16 weights, not for fp32 calls.  These (and
//    the scores of more than 8 rows a pass, where one conversion serves all
//    the rows) take n - 8 as a normal f16, two instructions per two elements.
//  - K's block scales multiply the fp32 block sums; V's multiply the softmax
//    weights before those are rounded to f16, with a running power-of-two
//    reference that keeps weight x scale below 2^14 and, for scales of usual
//    size, far above f16's smallest.
// Scores are S^T = K Q^T (16 tokens x 8 query rows per MMA), outputs O^T = V^T P^T
// (16 dims x 8 query rows): the query rows are the narrow side of both, so 8 rows
// fill them.  Between the two a tile's scores turn from a thread's (token, two
// rows) to (row, four tokens) through 1 KB of shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include <string>

#include "kvs.h"
#include "kvs_internal.h"

namespace kvs {
namespace {

constexpr int kTile = 32;          // tokens per tile (one bulk copy)
constexpr int kWarps = 4;          // warps per CTA; each works on its own
constexpr int kMaxSeq = 4096;      // sequences per call (their prefix sums live in shared memory)
constexpr int kMaxGroupRows = 64;  // n_rows * group bound
constexpr uint32_t kWaitLimit = 1u << 22;

using Pool = Q4Pool;

// ---------------------------------------------------------------- elements

__device__ __forceinline__ void put(void *p, int dtype, int64_t i, float x) {
    if (dtype == KVS_F32) static_cast<float *>(p)[i] = x;
    else if (dtype == KVS_F16) static_cast<__half *>(p)[i] = __float2half_rn(x);
    else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
}
__device__ __forceinline__ float2 two(uint32_t w, int dtype) {
    if (dtype == KVS_F16) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
}

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// ---------------------------------------------------------------- layout (include/kvs.h, "Q4 page layout")

__device__ __forceinline__ int k_word(int t, int b, int q, int NB) {  // byte offset of K bytes 4q .. 4q+3
    const int u = (t >> 3) * NB + b;
    return (((u >> 2) * 32) + (t & 7) * 4 + q) * 16 + (u & 3) * 4;
}
__device__ __forceinline__ int v_half(int t, int b, int j, int NB) {  // byte offset of V bytes j and j + 8 (j < 8)
    const int w = ((t >> 4) * NB + b) * 2 + ((t & 3) >> 1);
    return (((w >> 2) * 32) + j * 4 + ((t & 15) >> 2)) * 16 + (w & 3) * 4 + (t & 1) * 2;
}
__device__ __forceinline__ int k_scale(int t, int b, int NB) { return (((t >> 4) * 8 + (t & 7)) * NB + b) * 2 + (t >> 3 & 1); }
__device__ __forceinline__ int v_scale(int t, int b, int NB) { return ((t >> 2) * NB + b) * 4 + (t & 3); }

// ---------------------------------------------------------------- append / read
// Bound by bytes: rows at 2 or 4 bytes per element on one side, 9/16 byte on
// the other.  Four lanes share a 32-dim block, 8 dims each, so that rows are
// read and written in whole lines.  22161 rows of 4 x 256 bf16, 116 MB on both
// sides: read 25 us (4.6 TB/s); append 38 us (3.1 TB/s), bound by the
// instructions of the encoding and the wait for its rows, which 40 warps of 48
// registers hide best (53 us with both element sizes in one kernel of 64).

struct RowsParams {
    Pool pool;
    const int64_t *slots;
    int64_t n;
    const void *k, *v;
    void *ko, *vo;
    int64_t k_stride, v_stride;
    int dtype;
};

// 8 consecutive elements as they lie in memory, and as fp32
template <bool F32>
struct Eight {
    uint4 w[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        const uint4 *at = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p) + i * (F32 ? 4 : 2));
        w[0] = at[0];
        if (F32) w[F32 ? 1 : 0] = at[1];
    }
    __device__ __forceinline__ void zero() { w[0] = w[F32 ? 1 : 0] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(int dtype, float *x) const {
        if constexpr (F32) {
            x[0] = __uint_as_float(w[0].x), x[1] = __uint_as_float(w[0].y), x[2] = __uint_as_float(w[0].z), x[3] = __uint_as_float(w[0].w);
            x[4] = __uint_as_float(w[1].x), x[5] = __uint_as_float(w[1].y), x[6] = __uint_as_float(w[1].z), x[7] = __uint_as_float(w[1].w);
        } else {
            const float2 a = two(w[0].x, dtype), b = two(w[0].y, dtype), c = two(w[0].z, dtype), d = two(w[0].w, dtype);
            x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y, x[4] = c.x, x[5] = c.y, x[6] = d.x, x[7] = d.y;
        }
    }
};

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Q4_0 of a block whose dims 8 q .. 8 q + 7 lane q of its quad holds, in IEEE
// fp32 steps in a fixed order, the same as kvs_append's V: m = the element of
// largest |x| (lowest index on ties), d = m / -8, id = 1/d (0 if d == 0), code
// = trunc(x * id + 8.5) within 0 .. 15.  Lane q gets bytes 4 w .. 4 w + 3 of
// the block, w = 0, 2, 1, 3 for q = 0 .. 3.  (The kernels below are bound by
// instructions, so: m from the largest and the smallest element, in order only
// where those tie; x / -8 is x * -0.125; the code is read off the mantissa of
// the sum rounded down onto 2^23, two values an instruction.)
// x * id + 8.5, each rounded to nearest, then rounded down onto 2^23: a code in the low bits.  Two values an instruction.
// (The product is a multiply-add of 0: a plain multiply and the add after it may be joined into one rounding.)
__device__ __forceinline__ float2 scaled_rz(float2 x, float id) {
    float2 r;
    const float2 s = make_float2(id, id), h = make_float2(8.5f, 8.5f), big = make_float2(8388608.f, 8388608.f);
    asm("{\n .reg .b64 t;\n fma.rn.f32x2 t, %1, %2, %5;\n add.rn.f32x2 t, t, %3;\n add.rz.f32x2 %0, t, %4;\n}\n"
        : "=l"(*reinterpret_cast<uint64_t *>(&r))
        : "l"(*reinterpret_cast<const uint64_t *>(&x)), "l"(*reinterpret_cast<const uint64_t *>(&s)),
          "l"(*reinterpret_cast<const uint64_t *>(&h)), "l"(*reinterpret_cast<const uint64_t *>(&big)), "l"(0ull));
    return r;
}
__device__ __forceinline__ uint32_t q4_word(const float *x, int q, float &d) {
    float hi = max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), fmaxf(x[6], x[7]));
    float lo = min3(min3(x[0], x[1], x[2]), min3(x[3], x[4], x[5]), fminf(x[6], x[7]));
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    }
    float m = hi > -lo ? hi : lo;
    if (__any_sync(0xffffffffu, hi == -lo && hi != 0.f)) {  // both signs (some block of the warp): the first one decides
        int first = 32;
#pragma unroll
        for (int i = 7; i >= 0; --i)
            if (fabsf(x[i]) == hi) first = 8 * q + i;
        const int mine = first;
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
        float at = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (mine == 8 * q + i) at = x[i];
        at = __shfl_sync(0xffffffffu, at, (threadIdx.x & 28) + (first >> 3 & 3));
        if (hi == -lo) m = at;
    }
    d = __fmul_rn(m, -0.125f);
    const float id = (d != 0.0f) ? __frcp_rn(d) : 0.0f;
    uint32_t k[4];  // a code per half
    if (__any_sync(0xffffffffu, isinf(id))) {  // 1/d overflows below 2^-128: the other elements' codes are 0 or 15, 0 / d is 0's
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t c[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float u = fmaxf(__fadd_rn(__fmul_rn(x[2 * i + e], id), 8.5f), 0.f);
                c[e] = __float_as_uint(__fadd_rz(fminf(u, 15.f), 8388608.f)) & 15u;
            }
            k[i] = c[0] | c[1] << 16;
        }
    } else {  // x / d is within -8 .. 8 but for a rounding: the sum is positive and the code at most 16
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 r = scaled_rz(make_float2(x[2 * i], x[2 * i + 1]), id);
            k[i] = __vminu2(__byte_perm(__float_as_uint(r.x), __float_as_uint(r.y), 0x5410), 0x000f000fu);
        }
    }
    const uint32_t c[2] = {__byte_perm(k[0], k[1], 0x6420), __byte_perm(k[2], k[3], 0x6420)};  // a code per byte
    // lanes 0, 1 have the low nibbles of bytes 0-7, 8-15; lanes 2, 3 the high ones
    const uint32_t got = __shfl_xor_sync(0xffffffffu, q < 2 ? c[1] : c[0], 2);
    return q < 2 ? c[0] | got << 4 : got | c[1] << 4;
}
__device__ __forceinline__ int word_of(int q) { return q < 2 ? 2 * q : 2 * q - 3; }  // 0, 2, 1, 3

// K: one quad per (row, head, block), stored as it comes (a row's codes of one
// head are whole lines); kInFlight of them per thread, loaded before the first
// is encoded.
constexpr int kInFlight = 4;

// Where the 64 `each` (row, head, block or pair of blocks) units of a CTA lie: unit x of it is
// unit (rem + x) % per_row of row `row` + (rem + x) / per_row, in 32 bits.
struct Units {
    int64_t row;
    uint32_t rem, per_row;
    __device__ __forceinline__ Units(int64_t cta, int each, uint32_t per) : per_row(per) {
        const int64_t u = cta * (64 * each);
        row = u / per;
        rem = (uint32_t)(u - row * per);
    }
};

template <int D, bool F32>
__device__ void append_k(const RowsParams &p, int64_t block) {
    constexpr int NB = D / 32;
    const int q = threadIdx.x & 3;
    const Units units(block, kInFlight, NB * p.pool.Hk);
    int64_t row[kInFlight];
    uint32_t in_row[kInFlight];
    Eight<F32> x[kInFlight];
    int64_t slot[kInFlight];
#pragma unroll
    for (int m = 0; m < kInFlight; ++m) {
        const uint32_t u = units.rem + 64 * m + (threadIdx.x >> 2), r = u / units.per_row;
        row[m] = units.row + r;
        in_row[m] = u - r * units.per_row;
        slot[m] = row[m] < p.n ? p.slots[row[m]] : -1;
        if ((slot[m] >> p.pool.lgP) >= p.pool.n_pages) slot[m] = -1;
    }
#pragma unroll
    for (int m = 0; m < kInFlight; ++m) {
        x[m].zero();
        if (slot[m] >= 0) x[m].load(p.k, row[m] * p.k_stride + in_row[m] * 32 + 8 * q);
    }
#pragma unroll
    for (int m = 0; m < kInFlight; ++m) {
        const int b = in_row[m] % NB, h = in_row[m] / NB;
        float d, f[8];
        x[m].get(p.dtype, f);
        const uint32_t w = q4_word(f, q, d);
        if (slot[m] < 0) continue;
        const int tp = (int)(slot[m] & (p.pool.P - 1)), t = tp & 31;
        uint8_t *tile = p.pool.pages + (slot[m] >> p.pool.lgP) * p.pool.page_bytes + h * p.pool.head_bytes + (int64_t)(tp >> 5) * (36 * D);
        *reinterpret_cast<uint32_t *>(tile + k_word(t, b, word_of(q), NB)) = w;
        if (q == 0) reinterpret_cast<__half *>(tile + 16 * D)[k_scale(t, b, NB)] = __float2half_rn(d);
    }
}

// V: a byte of four tokens' codes makes up a 16-byte unit of the layout, so a
// CTA encodes 32 rows of a head (and up to 3 more) into shared memory and then
// stores units: groups of four consecutive rows that fill tokens 4 m .. 4 m + 3
// of a page, begun in the CTA's 32, whole; other rows two bytes at a time.
template <int D, bool F32>
__device__ void append_v(const RowsParams &p, int64_t chunk, int h) {
    constexpr int NB = D / 32, kRows = 32, kAll = kRows + 3, kPass = (kAll * NB + 63) / 64;
    __shared__ uint32_t code[kAll][NB * 4 + 1];  // padded: neighbouring rows on neighbouring banks
    __shared__ uint16_t scale[kAll][NB];
    __shared__ int64_t slot[kAll + 3];  // of rows i0 - 3 .. i0 + 34
    __shared__ int groups[9];           // rows at which whole groups begin; [8]: how many
    const int64_t i0 = chunk * kRows;
    const int tid = threadIdx.x, q = tid & 3;
    if (tid < kAll + 3) {
        const int64_t i = i0 - 3 + tid;
        const int64_t s = i >= 0 && i < p.n ? p.slots[i] : -1;
        slot[tid] = (s >> p.pool.lgP) < p.pool.n_pages ? s : -1;
    }
    __syncthreads();
    // whether row r (from i0) begins four rows that fill an aligned group of four tokens
    auto begins = [&](int r) {
        const int64_t s = slot[r + 3];
        return s >= 0 && (s & 3) == 0 && slot[r + 4] == s + 1 && slot[r + 5] == s + 2 && slot[r + 6] == s + 3;
    };
    const int rows = begins(kRows - 3) || begins(kRows - 2) || begins(kRows - 1) ? kAll : kRows;
    Eight<F32> v[kPass];
#pragma unroll
    for (int m = 0; m < kPass; ++m) {
        const int x = (tid >> 2) + 64 * m, r = x / NB, b = x % NB;
        v[m].zero();
        if (r < rows && i0 + r < p.n && slot[r + 3] >= 0) v[m].load(p.v, (i0 + r) * p.v_stride + (int64_t)h * D + b * 32 + 8 * q);
    }
    if (tid < 32) {
        const uint32_t at = __ballot_sync(0xffffffffu, begins(tid));
        if (begins(tid)) groups[__popc(at & ((1u << tid) - 1))] = tid;
        if (tid == 0) groups[8] = __popc(at);
    }
#pragma unroll
    for (int m = 0; m < kPass; ++m) {
        const int x = (tid >> 2) + 64 * m, r = x / NB, b = x % NB;
        if ((x & ~7) >= rows * NB) break;  // (the same in a warp)
        float d, f[8];
        v[m].get(p.dtype, f);
        const uint32_t w = q4_word(f, q, d);
        if (r < rows) {
            code[r][b * 4 + word_of(q)] = w;
            if (q == 0) scale[r][b] = __half_as_ushort(__float2half_rn(d));
        }
    }
    __syncthreads();
    auto tile_of = [&](int64_t s) {
        const int tp = (int)(s & (p.pool.P - 1));
        return p.pool.pages + (s >> p.pool.lgP) * p.pool.page_bytes + h * p.pool.head_bytes + (int64_t)(tp >> 5) * (36 * D);
    };
    // units: (group, block pair, j); neighbouring threads have neighbouring groups' units of one j
    for (int x = tid; x < 8 * (NB / 2) * 8; x += 256) {
        if ((x & 7) >= groups[8]) continue;
        const int r = groups[x & 7], j = x >> 3 & 7, bp = x >> 6;
        const int64_t s = slot[r + 3];
        const int t = (int)(s & 31);
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // word k: block 2 bp + k / 2, tokens 2 (k % 2) and + 1
            const int at = (2 * bp + (k >> 1)) * 4 + (j >> 2), ra = r + 2 * (k & 1);
            const uint32_t sel = (j & 3) | (uint32_t)(4 + (j & 3)) << 4;  // byte j and byte j + 8
            const uint32_t a0 = __byte_perm(code[ra][at], code[ra][at + 2], sel);
            const uint32_t a1 = __byte_perm(code[ra + 1][at], code[ra + 1][at + 2], sel);
            o[k] = (a0 & 0xffffu) | a1 << 16;
        }
        const int unit = (t >> 4) * (NB / 2) + bp;
        *reinterpret_cast<uint4 *>(tile_of(s) + 18 * D + (unit * 32 + j * 4 + ((t & 15) >> 2)) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    for (int x = tid; x < 8 * NB; x += 256) {
        const int b = x % NB;
        if (x / NB >= groups[8]) continue;
        const int r = groups[x / NB];
        const int64_t s = slot[r + 3];
        *reinterpret_cast<uint2 *>(tile_of(s) + 34 * D + v_scale((int)(s & 31), b, NB) * 2) =
            make_uint2(scale[r][b] | (uint32_t)scale[r + 1][b] << 16, scale[r + 2][b] | (uint32_t)scale[r + 3][b] << 16);
    }
    if (groups[8] == 8 && groups[0] == 0 && groups[7] == 28) return;  // they have every row
    for (int x = tid; x < kRows * NB * 8; x += 256) {  // rows of no whole group
        const int j = x & 7, b = (x >> 3) % NB, r = (x >> 3) / NB;
        const int64_t s = slot[r + 3];
        if (s < 0 || begins(r - (int)(s & 3))) continue;
        uint8_t *tile = tile_of(s);
        const int t = (int)(s & 31), at = b * 4 + (j >> 2);
        if (j == 0) reinterpret_cast<uint16_t *>(tile + 34 * D)[v_scale(t, b, NB)] = scale[r][b];
        const uint32_t lo = code[r][at] >> (8 * (j & 3)) & 0xff, hi = code[r][at + 2] >> (8 * (j & 3)) & 0xff;
        *reinterpret_cast<uint16_t *>(tile + 18 * D + v_half(t, b, j, NB)) = (uint16_t)(lo | hi << 8);
    }
}

// CTAs 0 .. k_blocks - 1 encode K, the others V (32 rows of a head each).
template <int D, bool F32>
__global__ void __launch_bounds__(256, F32 ? 3 : 5) append_kernel(const RowsParams p, int k_blocks) {
    if ((int)blockIdx.x < k_blocks) {
        append_k<D, F32>(p, blockIdx.x);
    } else {
        const int64_t c = blockIdx.x - k_blocks;
        append_v<D, F32>(p, c / p.pool.Hk, (int)(c % p.pool.Hk));
    }
}

// One quad per (row, head, pair of blocks): lanes q / 2 = 0 and 1 have a block
// each, and of it the dims 8 (q % 2) .. + 7 and the 8 that are 16 on, which are
// the low and the high nibbles of the same 8 bytes.  (With 8 dims of one block
// to a lane, its places worked out for half as many values: 29 us for 26 on the
// rows above; with four pairs in flight instead of two, as fast there and 20%
// slower on few rows.)
constexpr int kPairs = 2;  // per thread, loaded before the first is decoded
template <int D>
__global__ void __launch_bounds__(256) read_kernel(const RowsParams p) {
    constexpr int NB = D / 32;
    const bool is_v = blockIdx.y != 0;
    void *out = is_v ? p.vo : p.ko;
    if (!out) return;
    const int q = threadIdx.x & 3, side = q & 1;
    const Units units(blockIdx.x, kPairs, NB / 2 * p.pool.Hk);
    int64_t row[kPairs], slot[kPairs];
    uint32_t in_row[kPairs];
    uint32_t w[kPairs][2];  // bytes 8 side .. + 7 of the block; of V at first bytes j and j + 8 for j = 4 side .. + 3
    __half d[kPairs];
#pragma unroll
    for (int m = 0; m < kPairs; ++m) {
        const uint32_t u = units.rem + 64 * m + (threadIdx.x >> 2), r = u / units.per_row;
        row[m] = units.row + r;
        in_row[m] = u - r * units.per_row;
        slot[m] = row[m] < p.n ? p.slots[row[m]] : -1;
        if ((slot[m] >> p.pool.lgP) >= p.pool.n_pages) slot[m] = -1;
    }
#pragma unroll
    for (int m = 0; m < kPairs; ++m) {
        w[m][0] = w[m][1] = 0x88888888u;  // no slot: zeros
        d[m] = __ushort_as_half(0);
        if (slot[m] < 0) continue;
        const int b = in_row[m] % (NB / 2) * 2 + (q >> 1), h = in_row[m] / (NB / 2);
        const int tp = (int)(slot[m] & (p.pool.P - 1)), t = tp & 31;
        const uint8_t *tile = p.pool.pages + (slot[m] >> p.pool.lgP) * p.pool.page_bytes + h * p.pool.head_bytes + (int64_t)(tp >> 5) * (36 * D);
        if (!is_v) {
            const uint8_t *at = tile + k_word(t, b, 2 * side, NB);
            w[m][0] = *reinterpret_cast<const uint32_t *>(at);
            w[m][1] = *reinterpret_cast<const uint32_t *>(at + k_word(0, 0, 1, NB));
            d[m] = reinterpret_cast<const __half *>(tile + 16 * D)[k_scale(t, b, NB)];
        } else {
            const uint8_t *at = tile + 18 * D + v_half(t, b, 4 * side, NB);
            uint32_t x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = *reinterpret_cast<const uint16_t *>(at + v_half(0, 0, j, NB));
            w[m][0] = x[0] | x[1] << 16;
            w[m][1] = x[2] | x[3] << 16;
            d[m] = reinterpret_cast<const __half *>(tile + 34 * D)[v_scale(t, b, NB)];
        }
    }
#pragma unroll
    for (int m = 0; m < kPairs; ++m) {
        if (is_v) {  // the lane next to it has the other half of the low bytes and of the high ones
            const uint32_t low = __byte_perm(w[m][0], w[m][1], 0x6420u), high = __byte_perm(w[m][0], w[m][1], 0x7531u);
            const uint32_t got = __shfl_xor_sync(0xffffffffu, side ? low : high, 1);
            w[m][0] = side ? got : low;
            w[m][1] = side ? high : got;
        }
        if (row[m] >= p.n) continue;
        const int64_t at = (row[m] * units.per_row + in_row[m]) * 64 + 32 * (q >> 1) + 8 * side;
        // a nibble in the mantissa under exponent 0x64 is 1024 + n: minus 1032, exact; times the scale, rounded once
#pragma unroll
        for (int part = 0; part < 2; ++part) {  // dims 8 side .. + 7, then those + 16
            uint32_t code[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t nib = (part ? w[m][e] >> 4 : w[m][e]) & 0x0f0f0f0fu;
                code[2 * e] = hsub2(__byte_perm(nib, 0x64646464u, 0x4140), 0x64086408u);
                code[2 * e + 1] = hsub2(__byte_perm(nib, 0x64646464u, 0x4342), 0x64086408u);
            }
            uint32_t o[4];
            if (p.dtype == KVS_F16) {
                const __half2 s2 = __half2half2(d[m]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&code[e]), s2);
                    o[e] = *reinterpret_cast<const uint32_t *>(&v);
                }
            } else {
                const float s1 = __half2float(d[m]);
                float f[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&code[e]));
                    f[2 * e] = v.x * s1, f[2 * e + 1] = v.y * s1;
                }
                if (p.dtype == KVS_F32) {
                    float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(out) + at + 16 * part);
                    dst[0] = make_float4(f[0], f[1], f[2], f[3]);
                    dst[1] = make_float4(f[4], f[5], f[6], f[7]);
                    continue;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __nv_bfloat162 a = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
                    o[e] = *reinterpret_cast<const uint32_t *>(&a);
                }
            }
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at + 16 * part) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// ---------------------------------------------------------------- attention
// Work: the tiles of every (sequence, kv head) in one line, cut into equal
// contiguous ranges, one per warp ("worker"), whatever the sequences' lengths.
// A worker runs the online softmax over its tiles; where its range ends inside
// a (sequence, head) it leaves a partial (O, reference exponent, sum), at most
// two per worker, and the combine joins them in range order.  Query rows
// beyond one pass's 8 or 16 go to further workers over the same ranges, next
// to each other in the grid so that they share the tiles through L2.
// 32 sequences of 32768 .. 0 tokens, 32 / 8 heads, D 128, bf16: 90 us, 3.6 TB/s
// of the cache (55% of the measured copy rate), bound by the instructions of a
// tile, some 700 of a warp; with 4 rows each, 16 a pass, 146 us.  One of 4096
// tokens, 8 / 2 heads, fp32: 14 us, a chain of two launches.  Six of 65536 .. 0
// tokens, 24 / 4 heads, D 256, f16: 57 us for one row each (2.6 TB/s, 8 warps
// an SM), 121 for 4, whose 24 rows are three passes over the tiles.

struct AttendParams {
    Pool pool;
    const int32_t *table;
    const int32_t *lens;
    int64_t q_stride;
    const void *q;
    void *out;
    float *lse;
    float *part_o;   // [row block][worker][2][NT][2 D / 32][lane][4]: accumulators of 8 rows, see attend_kernel
    float2 *part_rl; // [row block][worker][2][NT][8]: reference exponent and sum of a row
    int table_width, n_seq, R, Hq, G;
    int dtype, row_blocks, workers;
    float scale_log2;
    int give_up;  // test hook: a worker's first wait gives up at once, as if its copy never landed
    int window, sinks;  // of the windowed kernels
};

__device__ __forceinline__ int seq_len(const Pool &pool, const int32_t *lens, int table_width, int s) {
    const int64_t cap = (int64_t)table_width << pool.lgP;
    const int n = lens[s];
    return n < 0 ? 0 : (int)(n < cap ? n : cap);
}

// Which tiles of a sequence of len tokens its rows see: all (WIN false), or
// under a window the first tokens' and those from the first row's window on:
// tile k of that line is k, or k + skip from `front` on.
// (So the work is cut over the tiles that count, and the masks are the two ends'
// alone: 32 sequences of up to 60000 tokens under a window of 4096, 32 / 8 heads,
// D 128, bf16, take 44 us for 113 MB, 2.6 TB/s: 8 for the two launches, the rest
// bound by the latency between a tile's dependent instructions, with half of the
// issue slots taken.  3.6 TB/s without a window, where the launches weigh less.)
template <bool WIN>
struct Seen {
    __device__ __forceinline__ Seen() {}
    __device__ __forceinline__ Seen(const AttendParams &, int) {}
    __device__ __forceinline__ int tiles(int len) const { return (len + kTile - 1) / kTile; }
    __device__ __forceinline__ int at(int k) const { return k; }
};
template <>
struct Seen<true> {
    int front, skip;
    __device__ __forceinline__ Seen() {}
    __device__ __forceinline__ Seen(const AttendParams &p, int len) {
        const int64_t from = (int64_t)len - p.R + 1 - p.window;  // the first row's window begins here
        const int first = from > 0 ? (int)(from / kTile) : 0, sink_tiles = (int)(((int64_t)p.sinks + kTile - 1) / kTile);
        front = sink_tiles < first ? sink_tiles : first;
        skip = first - front;
    }
    __device__ __forceinline__ int tiles(int len) const { return (len + kTile - 1) / kTile - skip; }
    __device__ __forceinline__ int at(int k) const { return k < front ? k : k + skip; }
};

// prefix[s] = {tiles of one head, sequences with tokens} of sequences 0 .. s-1;
// every thread of the CTA calls it
template <bool WIN = false>
__device__ void tile_prefix(const AttendParams &p, int2 *prefix) {
    const Pool &pool = p.pool;
    const int32_t *lens = p.lens;
    const int table_width = p.table_width, n_seq = p.n_seq;
    __shared__ int2 warp_sum[16];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
    const int per = (n_seq + nt - 1) / nt;
    int2 sum = make_int2(0, 0);
    for (int k = 0; k < per; ++k) {
        const int s = tid * per + k;
        if (s < n_seq) {
            const int len = seq_len(pool, lens, table_width, s), t = Seen<WIN>(p, len).tiles(len);
            sum.x += t;
            sum.y += t > 0;
        }
    }
    int2 inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc.x, o), y = __shfl_up_sync(0xffffffffu, inc.y, o);
        if (lane >= o) inc.x += x, inc.y += y;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int2 base = make_int2(inc.x - sum.x, inc.y - sum.y);
    for (int w = 0; w < warp; ++w) base.x += warp_sum[w].x, base.y += warp_sum[w].y;
    for (int k = 0; k < per; ++k) {
        const int s = tid * per + k;
        if (s < n_seq) {
            prefix[s] = base;
            const int len = seq_len(pool, lens, table_width, s), t = Seen<WIN>(p, len).tiles(len);
            base.x += t;
            base.y += t > 0;
        }
    }
    if (tid == nt - 1) prefix[n_seq] = base;
    __syncthreads();
}

// Ranges.  Beginning and ending a (sequence, head) costs a warp about as much
// as kHeadCost tiles (the query is fetched, results leave), so the line that is
// cut evenly is of cost: each (sequence, head) is kHeadCost units and its
// tiles.  (Cut by tiles alone, a worker with thirty one-tile heads took twice
// as long as all the others.)
constexpr int kHeadCost = 6;
constexpr int kMinTiles = 2;  // per worker, while that leaves some idle
// (The host refuses calls whose line could reach 2^31 units.)
struct Cut {
    uint32_t tiles, cost;  // in all
    uint32_t W, q, r;      // workers in use; units of each, and how many have one more
    __device__ __forceinline__ Cut(const int2 *prefix, int n_seq, int Hk, int workers) {
        tiles = (uint32_t)prefix[n_seq].x * Hk;
        cost = tiles + (uint32_t)(kHeadCost * prefix[n_seq].y * Hk);
        W = min((tiles + kMinTiles - 1) / kMinTiles, (uint32_t)workers);
        q = W ? cost / W : 0;
        r = cost - q * W;
    }
    __device__ __forceinline__ uint32_t begin(uint32_t w) const { return w * q + min(w, r); }  // cost unit at which worker w begins
    __device__ __forceinline__ int worker_of(uint32_t unit) const {
        const uint32_t cut = r * (q + 1);
        return (int)(unit < cut ? unit / (q + 1) : r + (unit - cut) / q);
    }
};
__device__ __forceinline__ uint32_t head_cost(int2 prefix, int Hk) { return (uint32_t)(prefix.x + kHeadCost * prefix.y) * Hk; }
// the last sequence whose tiles (cost) begin at or before `unit`
template <bool COST>
__device__ __forceinline__ int find_seq(const int2 *prefix, int n_seq, int Hk, uint32_t unit) {
    int lo = 0, hi = n_seq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((COST ? head_cost(prefix[mid], Hk) : (uint32_t)prefix[mid].x * Hk) <= unit) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}
// tiles before the cost unit `unit`
__device__ __forceinline__ uint32_t tiles_before(const int2 *prefix, int n_seq, int Hk, uint32_t unit, uint32_t all) {
    if (unit >= head_cost(prefix[n_seq], Hk)) return all;
    const int s = find_seq<true>(prefix, n_seq, Hk, unit);
    const uint32_t T = prefix[s + 1].x - prefix[s].x;
    const uint32_t in = unit - head_cost(prefix[s], Hk);
    const uint32_t h = in / (T + kHeadCost), o = in - h * (T + kHeadCost);
    return (uint32_t)prefix[s].x * Hk + h * T + (o > kHeadCost ? o - kHeadCost : 0);
}

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mma(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d = a * b + c, c kept
__device__ __forceinline__ void mma_from(float *d, const float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// the nearest multiple of 2^k, for c = 1.5 * 2^(23 + k) and |x| well below it
__device__ __forceinline__ float on_grid(float x, float c) { return __fadd_rn(__fadd_rn(x, c), -c); }
__device__ __forceinline__ float half_lo(uint32_t w) { return __low2float(*reinterpret_cast<const __half2 *>(&w)); }
__device__ __forceinline__ float half_hi(uint32_t w) { return __high2float(*reinterpret_cast<const __half2 *>(&w)); }

constexpr uint32_t kLoNib = 0x000f000fu, kHiNib = 0x00f000f0u;
constexpr uint32_t kLoOff = 0x00080008u, kHiOff = 0x00800080u;  // the offset 8 in place of a low and of a high nibble
// an ANDed nibble pair as the f16 numbers n - 8 (or 16 (n - 8)): under exponent 0x64 it is 1024 + n
__device__ __forceinline__ uint32_t centred(uint32_t nib, uint32_t off) { return hsub2(nib | 0x64006400u, off | 0x64006400u); }

// Query fragments of one pass: NT times 8 rows as the N side of the MMAs,
// fp32 queries as f16 hi + lo (HL).
template <int D, int NT, bool HL>
struct Query {
    static constexpr int NB = D / 32;
    // else the offset leaves the codes: one subtraction then serves NT row tiles, and sums of 0 .. 15 codes would leave
    // fp32 calls their own rounding
    static constexpr bool kBias = NT == 1 && !HL;
    uint32_t hi[NT][NB][2][2];              // row g: [block][k-step][low nibbles' dims, high nibbles' dims / 16]
    uint32_t lo[HL ? NT : 1][NB][2][2];
    float bias[kBias ? NB : 1][4];          // as an accumulator: -8 * 2^-24 * sum of the block's operands
    float fac[NT];                          // row g: accumulator -> log2 units (not negative)

    // The rows of (sequence, kv head) from rho0 on as they lie in memory: row rho
    // is query row rho / G, head h G + rho % G.  All loads are issued at once and
    // without a branch (a row past the last is the last one again).
    struct Raw {
        uint4 f[HL ? NT : 1][HL ? NB : 1][2];
        uint2 x[HL ? 1 : NT][HL ? 1 : NB][2];
        __device__ __forceinline__ void load(const AttendParams &p, int s, int h, int rho0) {
            const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int rho = min(rho0 + 8 * n + g, p.R * p.G - 1), r = rho / p.G;
                const int64_t base = ((int64_t)s * p.R + r) * p.q_stride + (int64_t)(h * p.G + rho - r * p.G) * D + 4 * t;
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if constexpr (HL) f[n][b][k] = *reinterpret_cast<const uint4 *>(static_cast<const float *>(p.q) + base + b * 32 + 16 * k);
                        else x[n][b][k] = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.q) + base + b * 32 + 16 * k);
                    }
            }
        }
        // dims 4t .. 4t + 3 (k = 0), 16 + 4t .. (k = 1) of block b
        __device__ __forceinline__ void get(int n, int b, int k, int dtype, float *y) const {
            if constexpr (HL) {
                const uint4 v = f[n][b][k];
                y[0] = __uint_as_float(v.x), y[1] = __uint_as_float(v.y), y[2] = __uint_as_float(v.z), y[3] = __uint_as_float(v.w);
            } else {
                const float2 a = two(x[n][b][k].x, dtype), c = two(x[n][b][k].y, dtype);
                y[0] = a.x, y[1] = a.y, y[2] = c.x, y[3] = c.y;
            }
        }
    };

    __device__ __forceinline__ void form(const AttendParams &p, const Raw &raw, int rho0) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const bool valid = rho0 + 8 * n + g < p.R * p.G;
            float top = 0.f;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float y[4];
                    raw.get(n, b, k, p.dtype, y);
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(y[i]));
                }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // a power of two that brings the row's largest element to 2^14 .. 2^15 (exact for
            // 16-bit elements down to 2^-28 of it; f16 then holds 2^-24 more below)
            int e = (int)(__float_as_uint(top) >> 23) - 127;
            e = e < -100 ? -100 : (e > 100 ? 100 : e);
            const float f = valid ? copysignf(__uint_as_float((uint32_t)(127 + 14 - e) << 23), p.scale_log2) : 0.f;
            // never 0, so that a masked score stays -inf times it (what a scale of 0, or one that vanishes here, takes
            // to 2^-126 instead is below 2^-80)
            fac[n] = fmaxf(fabsf(p.scale_log2) * __uint_as_float((uint32_t)(127 + (kBias ? 24 : 0) - 14 + e) << 23), 1.17549435e-38f);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float sum = 0.f, x[8];
                raw.get(n, b, 0, p.dtype, x);
                raw.get(n, b, 1, p.dtype, x + 4);
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    // k-step ks: low nibbles are dims 4t + ks and 4t + 2 + ks, high ones 16 further
                    float y[4] = {x[ks] * f, x[2 + ks] * f, x[4 + ks] * f, x[6 + ks] * f};
                    if constexpr (HL) {
                        // hi on a grid of 2^4 (2^11 steps of the row's largest element), so that its sums are exact in
                        // the tensor core, which cuts off products far below the largest; lo the rest
                        float z[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float h = on_grid(y[i], 201326592.f);  // 1.5 * 2^27
                            z[i] = y[i] - h;
                            y[i] = h;
                        }
                        lo[n][b][ks][0] = pack(z[0], z[1]);
                        lo[n][b][ks][1] = pack(z[2] * 0.0625f, z[3] * 0.0625f);
                    }
                    const uint32_t a0 = pack(y[0], y[1]), a1 = pack(y[2] * 0.0625f, y[3] * 0.0625f);
                    if constexpr (kBias) sum += half_lo(a0) + half_hi(a0) + 16.f * (half_lo(a1) + half_hi(a1));
                    hi[n][b][ks][0] = a0;
                    hi[n][b][ks][1] = a1;
                }
                if constexpr (kBias) {
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                    sum *= -8.f * 5.9604644775390625e-8f;
                    bias[b][0] = bias[b][2] = __shfl_sync(0xffffffffu, sum, 8 * t);
                    bias[b][1] = bias[b][3] = __shfl_sync(0xffffffffu, sum, 8 * t + 4);
                    // (four registers, ready to be an MMA's C: the compiler would fold the pairs and copy them each time)
                    asm volatile("" : "+f"(bias[b][0]), "+f"(bias[b][1]), "+f"(bias[b][2]), "+f"(bias[b][3]));
                }
            }
        }
    }

    // scores, not yet times fac, of the tile's tokens 16 c + g and 16 c + 8 + g:
    // acc[n] = {(g, row 2t), (g, row 2t + 1), (g + 8, row 2t), (g + 8, row 2t + 1)}
    __device__ __forceinline__ void scores(const uint8_t *tile, int c, float (*acc)[4]) const {
        const int lane = threadIdx.x & 31, g = lane >> 2;
        const uint8_t *ps = tile + 16 * D + (c * 8 + g) * NB * 4;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
        constexpr int kGroup = NB < 4 ? NB : 4;  // blocks fetched together
#pragma unroll
        for (int b0 = 0; b0 < NB; b0 += kGroup) {
            uint32_t sc[kGroup], w[2][kGroup];
            if constexpr (NB == 2) {
                const uint2 v = *reinterpret_cast<const uint2 *>(ps);
                sc[0] = v.x, sc[1] = v.y;
                const uint4 k = *reinterpret_cast<const uint4 *>(tile + (c * 32 + lane) * 16);
                w[0][0] = k.x, w[0][1] = k.y, w[1][0] = k.z, w[1][1] = k.w;
            } else {
                const uint4 v = *reinterpret_cast<const uint4 *>(ps + b0 * 4);
                sc[0] = v.x, sc[1] = v.y, sc[2] = v.z, sc[3] = v.w;
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    const uint4 k = *reinterpret_cast<const uint4 *>(tile + (((2 * c + o) * (NB / 4) + b0 / 4) * 32 + lane) * 16);
                    w[o][0] = k.x, w[o][1] = k.y, w[o][2] = k.z, w[o][3] = k.w;
                }
            }
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {
                const int b = b0 + i;
                const uint32_t x0 = w[0][i] >> 8, x1 = w[1][i] >> 8;
                uint32_t a0 = w[0][i] & kLoNib, a1 = w[1][i] & kLoNib, a2 = w[0][i] & kHiNib, a3 = w[1][i] & kHiNib;
                uint32_t e0 = x0 & kLoNib, e1 = x1 & kLoNib, e2 = x0 & kHiNib, e3 = x1 & kHiNib;
                if constexpr (!kBias) {
                    a0 = centred(a0, kLoOff), a1 = centred(a1, kLoOff), a2 = centred(a2, kHiOff), a3 = centred(a3, kHiOff);
                    e0 = centred(e0, kLoOff), e1 = centred(e1, kLoOff), e2 = centred(e2, kHiOff), e3 = centred(e3, kHiOff);
                }
                const float s0 = half_lo(sc[i]), s1 = half_hi(sc[i]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float d[4];
                    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_from(d, kBias ? bias[kBias ? b : 0] : zero, a0, a1, a2, a3, hi[n][b][0][0], hi[n][b][0][1]);
                    mma(d, e0, e1, e2, e3, hi[n][b][1][0], hi[n][b][1][1]);
                    if constexpr (HL) {  // summed apart, below the cut of hi's sums
                        float r[4];
                        mma_from(r, zero, a0, a1, a2, a3, lo[n][b][0][0], lo[n][b][0][1]);
                        mma(r, e0, e1, e2, e3, lo[n][b][1][0], lo[n][b][1][1]);
#pragma unroll
                        for (int k = 0; k < 4; ++k) d[k] += r[k];
                    }
                    acc[n][0] = fmaf(d[0], s0, acc[n][0]);
                    acc[n][1] = fmaf(d[1], s0, acc[n][1]);
                    acc[n][2] = fmaf(d[2], s1, acc[n][2]);
                    acc[n][3] = fmaf(d[3], s1, acc[n][3]);
                }
            }
        }
    }
};

// Row r's scores of a tile in shared memory: 32 floats, its 16-byte chunk c at
// place c ^ turn(r).  Writes (rows 2t or 2t + 1, tokens g) and reads (rows g,
// chunks t) of a warp both hit every bank once.
__device__ __forceinline__ int turn(int r) { return (r & 6) ^ ((r & 1) << 2); }

// A power of two above the V scales a worker has met in a (sequence, head), by
// the highest bit that any of their exponent fields has set: the field is below
// 16, 8, 4, 2 or 1, so that one OR of the packed scales and one AND test them.
// (Scales of 2 and more share that bit and are bounded one by one.)
struct ScaleBound {
    uint32_t over;  // exponent bits (of both halves) that no scale so far has; all ones: no scale yet
    float lg;       // |scale| < 2^lg
    __device__ __forceinline__ void reset() {
        over = ~0u;
        lg = -14.f;
    }
    // bits: the OR of scales over the warp; most: of this lane's scales the largest (for those of 2 and more)
    __device__ __forceinline__ void raise(uint32_t bits, float most) {
        const uint32_t e = (bits | bits >> 16) & 0x7c00u;
        float to = e & 0x2000u ? 1.f : e & 0x1000u ? -7.f : e & 0x0800u ? -11.f : e & 0x0400u ? -13.f : -14.f;
        uint32_t o = e & 0x2000u ? 0x4000u : e & 0x1000u ? 0x6000u : e & 0x0800u ? 0x7000u : e & 0x0400u ? 0x7800u : 0x7c00u;
        if (e & 0x4000u) {
#pragma unroll
            for (int k = 16; k; k >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, k));
            to = fminf(fmaxf((float)((int)(__float_as_uint(most) >> 23) - 126), 1.f), 16.f);  // (f16 ends below 2^16)
            o = 0x4000u;
        }
        if (to >= lg) {
            lg = to;
            over = o | o << 16;
        }
    }
};

// A warp's stages in shared memory and the bulk copies into them.
template <int BYTES, int NST>
struct Stages {
    uint32_t bar0, buf0;
    const uint8_t *buf;
    uint32_t bad;   // stage holds no tile: its page number was outside the pool
    bool gave_up;

    __device__ __forceinline__ void init(uint8_t *smem, uint64_t *bars) {
        buf = smem;
        buf0 = smem_addr(smem);
        bar0 = smem_addr(bars);
        bad = 0;
        gave_up = false;
        if ((threadIdx.x & 31) == 0) {
            for (int i = 0; i < NST; ++i)
                asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar0 + 8 * i));
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
    }
    __device__ __forceinline__ void fetch(int stage, const uint8_t *src) {  // src null: a bad page (warp-uniform)
        if (!src) {
            bad |= 1u << stage;
            return;
        }
        bad &= ~(1u << stage);
        if ((threadIdx.x & 31) == 0) {
            const uint32_t bar = bar0 + 8 * stage;
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(BYTES) : "memory");
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                    buf0 + stage * BYTES),
                "l"(src), "r"(BYTES), "r"(bar)
                : "memory");
        }
    }
    // whether the copy into a stage that completes the phase of this parity lands in time
    __device__ __forceinline__ bool landed(int stage, uint32_t parity) const {
        uint32_t done = 0;
        if ((threadIdx.x & 31) == 0)  // one lane polls: a poll by 32 lanes holds the warp for 200 clocks
            for (uint32_t i = 0; i < kWaitLimit && !done; ++i)
                asm volatile(
                    "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
                    : "=r"(done)
                    : "r"(bar0 + 8 * stage), "r"(parity)
                    : "memory");
        done = __shfl_sync(0xffffffffu, done, 0);
        __syncwarp();  // what lane 0 saw complete, the others may read
        return done != 0;
    }
    // the stage's tile, or false: bad page, or the copy never landed.  phases: per stage the parity of its next wait.
    __device__ __forceinline__ bool wait(int stage, uint32_t &phases) {
        if (gave_up || (bad >> stage & 1)) return false;
        const uint32_t parity = phases >> stage & 1;
        phases ^= 1u << stage;
        gave_up = !landed(stage, parity);
        return !gave_up;
    }
    // what a wait on `stage` that gives up leaves (test hook)
    __device__ __forceinline__ void give_up(int stage, uint32_t &phases) {
        phases ^= 1u << stage;
        gave_up = true;
    }
    // After the wait on stage `first` gave up: its copy and those of the stages after it, n in all, were begun and not seen
    // to land; they still write this CTA's shared memory.  Each gets the whole time again, whatever became of the one before.
    __device__ __forceinline__ void drain(int first, int n, uint32_t phases) const {
        phases ^= 1u << first;  // (turned by the wait that gave up)
        for (int i = 0, s = first; i < n; ++i, s = s + 1 == NST ? 0 : s + 1)
            if (!(bad >> s & 1)) landed(s, phases >> s & 1);
    }
};

// A place in the line of tiles: tile k of T of (sequence, head).
struct Place {
    int s, h, k, T;
    __device__ __forceinline__ bool next(const int2 *prefix, int n_seq, int Hk) {  // whether (s, h) changed
        if (++k < T) return false;
        k = 0;
        if (++h < Hk) return true;
        h = 0;
        do {
            ++s;
        } while (s < n_seq && prefix[s + 1].x == prefix[s].x);
        if (s >= n_seq) {  // past the last tile: never fetched
            s = n_seq - 1;
            T = 1 << 30;
            return false;
        }
        T = prefix[s + 1].x - prefix[s].x;
        return true;
    }
};

// The same with the pages ahead, for the copies.
template <bool WIN = false>
struct Cursor : Place {
    int page_base, page;  // lane l holds page number page_base + l of the sequence
    int page_at;          // the page (of the sequence) that base points into; -1: none yet
    const uint8_t *base;
    Seen<WIN> seen;
    __device__ __forceinline__ void load_pages(const AttendParams &p, int tiles_per_page_lg) {
        const int lane = threadIdx.x & 31;
        page_base = seen.at(k) >> tiles_per_page_lg;
        page_at = -1;
        const int at = page_base + lane;
        page = at < p.table_width ? p.table[(int64_t)s * p.table_width + at] : -1;
    }
    __device__ __forceinline__ void begin(const AttendParams &p, int lg) {  // of a (sequence, head)
        if constexpr (WIN) seen = Seen<WIN>(p, seq_len(p.pool, p.lens, p.table_width, s));
        load_pages(p, lg);
    }
    __device__ __forceinline__ void seek(const AttendParams &p, const int2 *prefix, uint32_t unit, int lg) {
        s = find_seq<false>(prefix, p.n_seq, p.pool.Hk, unit);
        T = prefix[s + 1].x - prefix[s].x;
        const uint32_t in = unit - (uint32_t)prefix[s].x * p.pool.Hk;
        h = (int)(in / (uint32_t)T);
        k = (int)(in - (uint32_t)h * (uint32_t)T);
        begin(p, lg);
    }
    // the tile's bytes (null: a page number outside the pool), warp-uniform
    __device__ __forceinline__ const uint8_t *tile(const AttendParams &p, int lg, int tile_bytes) {
        const int kt = seen.at(k), at = kt >> lg;
        if (at != page_at) {
            if (at - page_base >= 32) load_pages(p, lg);
            const int pg = __shfl_sync(0xffffffffu, page, at - page_base);
            base = pg < 0 || pg >= p.pool.n_pages ? nullptr : p.pool.pages + pg * p.pool.page_bytes + h * p.pool.head_bytes;
            page_at = at;
        }
        return base ? base + (kt & ((1 << lg) - 1)) * tile_bytes : nullptr;
    }
    __device__ __forceinline__ void advance(const AttendParams &p, const int2 *prefix, int lg) {
        if (next(prefix, p.n_seq, p.pool.Hk)) begin(p, lg);
    }
};

template <int D>
__host__ __device__ constexpr int stages_of() {
    return D == 64 ? 4 : 3;
}
// bytes per warp for turned scores beyond the tile's own
__host__ __device__ constexpr int turn_bytes(int D, int NT) { return NT * 1024 > 8 * D ? NT * 1024 : 0; }
// CTAs of an SM.  A warp's tile takes it some 3000 clocks whatever the others
// do, so what counts is how many warps the registers allow without spills: 16
// at 128 registers each (D = 64), 12 at 168 (D = 128; 16 that spill: 95 us for
// 12's 89), 8 at 255.  (Shared memory allows as many up to some 600 sequences:
// their prefix sums are 8 bytes each.  At D = 256 a larger batch has one CTA.)
__host__ __device__ constexpr int attend_ctas(int D, int NT) { return D == 256 ? 2 : (D == 128 || NT == 2 ? 3 : 4); }
template <int D, int NT, bool HL, bool WIN>
__global__ void __launch_bounds__(kWarps * 32, attend_ctas(D, NT)) attend_kernel(const AttendParams p) {
    constexpr int NB = D / 32, NST = stages_of<D>(), BYTES = 36 * D, kTurnBytes = turn_bytes(D, NT);
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[kWarps * NST];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    int2 *prefix = reinterpret_cast<int2 *>(smem + kWarps * (NST * BYTES + kTurnBytes));
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tile_prefix<WIN>(p, prefix);
    const Cut cut(prefix, p.n_seq, p.pool.Hk, p.workers);
    const int rb = blockIdx.x % p.row_blocks;
    const int w = (int)(blockIdx.x / p.row_blocks) * kWarps + warp;
    if (w >= (int)cut.W) return;
    const uint32_t u0 = tiles_before(prefix, p.n_seq, p.pool.Hk, cut.begin(w), cut.tiles);
    const uint32_t u1 = tiles_before(prefix, p.n_seq, p.pool.Hk, cut.begin(w + 1), cut.tiles);
    if (u0 >= u1) return;
    const int lg = p.pool.lgP - 5;
    const int rho0 = rb * 8 * NT;

    Stages<BYTES, NST> st;
    st.init(smem + warp * NST * BYTES, bars + warp * NST);
    uint32_t phases = 0;
    Cursor<WIN> ahead;
    ahead.seek(p, prefix, u0, lg);
    Place at = ahead;
    const int units = (int)(u1 - u0);
    int fetched = 0;
#pragma unroll
    for (int i = 0; i < NST; ++i) {
        if (fetched < units) {
            st.fetch(i, ahead.tile(p, lg, BYTES));
            ahead.advance(p, prefix, lg);
            ++fetched;
        }
    }
    Query<D, NT, HL> q;
    // cs: block b's -8 * 2^-24 * sum p s, in an accumulator of its own or in row b of one
    constexpr float kUnit = HL ? 1.f : 16777216.f;  // V's codes are subnormal, or n - 8 as it stands
    constexpr bool kOwnSum = NT == 1 && D <= 128;
    constexpr int kSums = kOwnSum ? NB : 1;
    float O[NT][NB][2][4], cs[NT][kSums][4], ref[NT], l[NT];
    bool fresh = true;
    int k_first = 0, len = 0;
    Seen<WIN> seen;
    ScaleBound bound;
    int stage = 0, unit = 0;
    if (p.give_up) st.give_up(stage, phases);
    for (; unit < units; ++unit) {
        if (fresh) {  // a new (sequence, head)
            typename Query<D, NT, HL>::Raw raw;
            raw.load(p, at.s, at.h, rho0);  // the tiles' copies are under way
            len = seq_len(p.pool, p.lens, p.table_width, at.s);
            if constexpr (WIN) seen = Seen<WIN>(p, len);
            q.form(p, raw, rho0);
            k_first = at.k;
            bound.reset();
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                ref[n] = -INFINITY;
                l[n] = 0.f;
#pragma unroll
                for (int b = 0; b < kSums; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) cs[n][b][i] = 0.f;
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) O[n][b][0][i] = O[n][b][1][i] = 0.f;
            }
            fresh = false;
        }
        if (!st.wait(stage, phases)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) l[n] = __int_as_float(0x7fc00000);
            if (st.gave_up) break;
        } else {
            const uint8_t *tile = st.buf + stage * BYTES;
            // the turned scores (1 KB per 8 rows) take the place of the K codes that are read first, where those are as
            // many bytes (8 D), else an area of their own
            float *turned = reinterpret_cast<float *>(kTurnBytes ? smem + kWarps * NST * BYTES + warp * kTurnBytes : const_cast<uint8_t *>(tile));
            const int in_tile = len - seen.at(at.k) * kTile;  // tokens of the sequence from this tile on
            // Scores, 16 tokens at a time, into the turned tile.  (With 16 rows a pass the loops over the halves stay
            // rolled: unrolled, the live values exceed the registers, 237 against 175 us.)
            constexpr int kUnroll = NT == 1 ? 2 : 1;
#pragma unroll kUnroll
            for (int c = 0; c < 2; ++c) {
                float acc[NT][4];
                q.scores(tile, c, acc);
                __syncwarp();  // the K codes of these tokens have been read by every lane
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = 2 * t + (i & 1), tok = 16 * c + 8 * (i >> 1) + g;
                        turned[n * 256 + row * 32 + (((tok >> 2) ^ turn(row)) << 2) + (tok & 3)] = acc[n][i];
                    }
            }
            __syncwarp();
            // row g, tokens 16 c + 4 t + (0 .. 3), not yet times fac; -inf for those the row does not see
            const bool masked = in_tile - (p.R - 1) < kTile;
            // the last row's window begins behind this tile's first token, and not all of it is of the first that stay
            const bool behind = WIN && in_tile > p.window && len - in_tile + kTile > p.sinks;
            auto row_scores = [&](int n, int c, float *x) {
                const float4 v = *reinterpret_cast<const float4 *>(turned + n * 256 + g * 32 + (((4 * c + t) ^ turn(g)) << 2));
                x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
                if (masked) {
                    const int see = in_tile - (p.R - 1) + (rho0 + 8 * n + g) / p.G - 16 * c - 4 * t;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i >= see) x[i] = -INFINITY;
                }
                if constexpr (WIN) {
                    if (behind) {
                        const int at0 = 16 * c + 4 * t, from = in_tile - p.R + (rho0 + 8 * n + g) / p.G + 1 - p.window - at0;
                        const int stay = p.sinks - (len - in_tile) - at0;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (i < from && i >= stay) x[i] = -INFINITY;
                    }
                }
            };
            if (bound.over == ~0u) {  // the head's first tile sets the bound
                uint32_t any = 0;
#pragma unroll
                for (int i = lane; i < NB * 8; i += 32) {
                    uint2 v = reinterpret_cast<const uint2 *>(tile + 34 * D)[i];
                    const int left = in_tile - 4 * (i / NB);  // of its four tokens
                    if (left < 4) {
                        v.x &= (left > 0 ? 0xffffu : 0u) | (left > 1 ? 0xffff0000u : 0u);
                        v.y &= left > 2 ? 0xffffu : 0u;
                    }
                    any |= v.x | v.y;
                }
                bound.raise(__reduce_or_sync(0xffffffffu, any), 0.f);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float x[8];
                row_scores(n, 0, x);
                row_scores(n, 1, x + 4);
                float mx = max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), fmaxf(x[6], x[7]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                // weight x scale is below 2^(need - ref): kept at 2^14 at most
                const float need = mx * q.fac[n] + bound.lg;
                const bool grow = need - 14.f > ref[n];
                if (__any_sync(0xffffffffu, grow)) {
                    const float to = grow ? need - 8.f : ref[n];
                    const float alpha = ref[n] == -INFINITY ? 0.f : exp2f(ref[n] - to);
                    ref[n] = to;
                    l[n] *= alpha;
                    const float a0 = __shfl_sync(0xffffffffu, alpha, 8 * t), a1 = __shfl_sync(0xffffffffu, alpha, 8 * t + 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float al = (i & 1) ? a1 : a0;
#pragma unroll
                        for (int b = 0; b < kSums; ++b) cs[n][b][i] *= al;
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            O[n][b][0][i] *= al;
                            O[n][b][1][i] *= al;
                        }
                    }
                }
            }
            // O^T += V^T (p s)^T, 16 tokens and two blocks at a time
#pragma unroll kUnroll
            for (int c = 0; c < 2; ++c) {
                float x[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    row_scores(n, c, x[n]);
                    const float r0 = ref[n] == -INFINITY ? 0.f : ref[n];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[n][i] = ex2(fmaf(x[n][i], q.fac[n], -r0));
                        l[n] += x[n][i];
                    }
                }
#pragma unroll
                for (int b0 = 0; b0 < NB; b0 += 2) {
                    const uint4 sv = *reinterpret_cast<const uint4 *>(tile + 34 * D + ((c * 4 + t) * NB + b0) * 8);
                    const uint4 vw = *reinterpret_cast<const uint4 *>(tile + 18 * D + ((c * (NB / 2) + b0 / 2) * 32 + lane) * 16);
                    uint32_t vs[2][2] = {{sv.x, sv.y}, {sv.z, sv.w}};  // [block]: tokens 16 c + 4 t + (0, 1), (2, 3)
                    if (in_tile < kTile) {  // scales of tokens never written may be anything and count as 0
                        const int left = in_tile - 16 * c - 4 * t;
                        const uint32_t k0 = (left > 0 ? 0xffffu : 0u) | (left > 1 ? 0xffff0000u : 0u);
                        const uint32_t k1 = (left > 2 ? 0xffffu : 0u) | (left > 3 ? 0xffff0000u : 0u);
                        vs[0][0] &= k0, vs[1][0] &= k0, vs[0][1] &= k1, vs[1][1] &= k1;
                    }
                    // a scale beyond the bound kept so far (rare): everything so far is brought to the larger one
                    const uint32_t any = vs[0][0] | vs[0][1] | vs[1][0] | vs[1][1];
                    if (__any_sync(0xffffffffu, any & bound.over)) {
                        float most = 0.f;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            most = fmaxf(most, fmaxf(fabsf(half_lo(vs[i >> 1][i & 1])), fabsf(half_hi(vs[i >> 1][i & 1]))));
                        const float was = bound.lg;
                        bound.raise(__reduce_or_sync(0xffffffffu, any), most);
                        const float up = bound.lg - was;
                        if (up > 0.f) {
                            const float f = __uint_as_float((uint32_t)(127 - (int)up) << 23);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                ref[n] += up;
                                l[n] *= f;
#pragma unroll
                                for (int i = 0; i < 4; ++i) x[n][i] *= f;
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
#pragma unroll
                                    for (int b = 0; b < kSums; ++b) cs[n][b][i] *= f;
#pragma unroll
                                    for (int b = 0; b < NB; ++b) O[n][b][0][i] *= f, O[n][b][1][i] *= f;
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int b = b0 + i;
                        const float s0 = half_lo(vs[i][0]), s1 = half_hi(vs[i][0]), s2 = half_lo(vs[i][1]), s3 = half_hi(vs[i][1]);
                        const uint32_t w0 = i ? vw.z : vw.x, w1 = i ? vw.w : vw.y;
                        uint32_t a0 = w0 & kLoNib, a1 = w0 & kHiNib, a2 = w1 & kLoNib, a3 = w1 & kHiNib;
                        uint32_t e0 = (w0 >> 8) & kLoNib, e1 = (w0 >> 8) & kHiNib, e2 = (w1 >> 8) & kLoNib, e3 = (w1 >> 8) & kHiNib;
                        if constexpr (HL) {
                            a0 = centred(a0, kLoOff), a2 = centred(a2, kLoOff), a1 = centred(a1, kHiOff), a3 = centred(a3, kHiOff);
                            e0 = centred(e0, kLoOff), e2 = centred(e2, kLoOff), e1 = centred(e1, kHiOff), e3 = centred(e3, kHiOff);
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const float y0 = x[n][0] * s0, y1 = x[n][1] * s1, y2 = x[n][2] * s2, y3 = x[n][3] * s3;
                            const uint32_t p0 = pack(y0, y1), p1 = pack(y2, y3);
                            mma(O[n][b][0], a0, a1, a2, a3, p0, p1);
                            mma(O[n][b][1], e0, e1, e2, e3, p0, p1);
                            if constexpr (HL) {
                                const uint32_t d0 = pack(y0 - half_lo(p0), y1 - half_hi(p0)), d1 = pack(y2 - half_lo(p1), y3 - half_hi(p1));
                                mma(O[n][b][0], a0, a1, a2, a3, d0, d1);
                                mma(O[n][b][1], e0, e1, e2, e3, d0, d1);
                            } else if constexpr (kOwnSum) {  // -8 * 2^-24 (f16 subnormal) times the sum of the same operands
                                constexpr uint32_t eight = kLoOff | 0x80008000u;
                                mma(cs[n][b], eight, eight, eight, eight, p0, p1);
                            } else {  // the same in row b
                                const uint32_t eight = g == b ? kLoOff | 0x80008000u : 0u;
                                mma(cs[n][0], eight, 0u, eight, 0u, p0, p1);
                            }
                        }
                    }
                }
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the turned scores, before a copy over them
        __syncwarp();
        const bool last_of_head = at.k + 1 == at.T;
        if (fetched < units) {
            st.fetch(stage, ahead.tile(p, lg, BYTES));
            ahead.advance(p, prefix, lg);
            ++fetched;
        }
        stage = stage + 1 == NST ? 0 : stage + 1;
        if (last_of_head || unit + 1 == units) {
            const bool whole = k_first == 0 && last_of_head;
            const int slot = unit == at.k - k_first ? 0 : 1;  // the worker's first (sequence, head), or its last
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                l[n] += __shfl_xor_sync(0xffffffffu, l[n], 1);
                l[n] += __shfl_xor_sync(0xffffffffu, l[n], 2);
                const float l0 = __shfl_sync(0xffffffffu, l[n], 8 * t), l1 = __shfl_sync(0xffffffffu, l[n], 8 * t + 4);
                // a row that saw nothing: out 0, lse -inf
                const float i0 = whole ? (l0 == 0.f ? 0.f : 1.f / l0) : 1.f, i1 = whole ? (l1 == 0.f ? 0.f : 1.f / l1) : 1.f;
                float off[NB][2];  // of rows 2t, 2t + 1
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        off[b][c] = kOwnSum ? cs[n][kOwnSum ? b : 0][c] : __shfl_sync(0xffffffffu, cs[n][0][c], b * 4 + t);
                if (!whole) {  // the accumulators as they are, 16 bytes a lane
                    const int64_t pslot = (((int64_t)rb * p.workers + w) * 2 + slot) * NT + n;
                    float4 *dst = reinterpret_cast<float4 *>(p.part_o) + pslot * (2 * NB * 32) + lane;
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int m = 0; m < 2; ++m)
                            dst[(2 * b + m) * 32] = make_float4((O[n][b][m][0] + off[b][0]) * kUnit, (O[n][b][m][1] + off[b][1]) * kUnit,
                                                                (O[n][b][m][2] * 0.0625f + off[b][0]) * kUnit,
                                                                (O[n][b][m][3] * 0.0625f + off[b][1]) * kUnit);
                    if (t == 0) p.part_rl[pslot * 8 + g] = make_float2(ref[n], l[n]);
                    continue;
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int rho = rho0 + 8 * n + 2 * t + c;
                    const float inv = (c ? i1 : i0) * kUnit;
                    if (rho >= p.R * p.G) continue;
                    const int64_t orow = (((int64_t)at.s * p.R + rho / p.G) * p.Hq + at.h * p.G + rho % p.G) * D;
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const int dim = b * 32 + 8 * m + g;
                            put(p.out, p.dtype, orow + dim, (O[n][b][m][c] + off[b][c]) * inv);
                            put(p.out, p.dtype, orow + dim + 16, (O[n][b][m][2 + c] * 0.0625f + off[b][c]) * inv);
                        }
                }
                const int rho = rho0 + 8 * n + g;
                if (t == 0 && rho < p.R * p.G && p.lse)
                    p.lse[((int64_t)at.s * p.R + rho / p.G) * p.Hq + at.h * p.G + rho % p.G] =
                        l[n] == 0.f ? -INFINITY : (ref[n] + log2f(l[n])) * 0.693147180559945309f;
            }
            fresh = true;
        }
        at.next(prefix, p.n_seq, p.pool.Hk);
    }
    if (st.gave_up) {  // what this worker owed is NaN: partials and whole rows of its range
        st.drain(stage, fetched - unit, phases);
        for (int i = lane; i < 2 * 8 * NT; i += 32)
            p.part_rl[((int64_t)rb * p.workers + w) * 2 * (8 * NT) + i] = make_float2(0.f, __int_as_float(0x7fc00000));  // (the sum: NaN)
        Cursor<WIN> c;
        c.seek(p, prefix, u0, lg);
        for (int x = 0; x < units; ++x) {
            if (c.k == 0 && x + c.T <= units)
                for (int rho = rho0; rho < rho0 + 8 * NT && rho < p.R * p.G; ++rho) {
                    const int64_t row = ((int64_t)c.s * p.R + rho / p.G) * p.Hq + c.h * p.G + rho % p.G;
                    for (int d = lane; d < D; d += 32) put(p.out, p.dtype, row * D + d, __int_as_float(0x7fc00000));
                    if (lane == 0 && p.lse) p.lse[row] = __int_as_float(0x7fc00000);
                }
            c.next(prefix, p.n_seq, p.pool.Hk);
        }
    }
}

// One CTA per (sequence, kv head, 8 rows of a pass, 64 dims): joins the
// partials of a (sequence, head) that several workers shared, its warps each a
// part of them, in the accumulators' own layout; rows of empty sequences are
// written here.
constexpr int kJoinVecs = 4;    // of the 2 D / 32 vectors of a partial: 64 dims
constexpr int kJoinAtOnce = 4;  // partials a warp has on their way
template <int D, int kJoinWarps, bool WIN>
__global__ void __launch_bounds__(kJoinWarps * 32) combine_kernel(const AttendParams p, int nt) {
    constexpr int kVec = 2 * D / 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float4 part[kJoinWarps][kJoinVecs * 32];
    __shared__ float sums[kJoinWarps][8], refs[8];
    int2 *prefix = reinterpret_cast<int2 *>(smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    tile_prefix<WIN>(p, prefix);
    const Cut cut(prefix, p.n_seq, p.pool.Hk, p.workers);
    const int rows = p.R * p.G, groups = (rows + 7) / 8, v0 = blockIdx.y * kJoinVecs, d0 = v0 * 16;
    const int grp = blockIdx.x % groups, h = blockIdx.x / groups % p.pool.Hk, s = blockIdx.x / groups / p.pool.Hk;
    const int T = prefix[s + 1].x - prefix[s].x;
    auto row_at = [&](int rho) { return ((int64_t)s * p.R + rho / p.G) * p.Hq + h * p.G + rho % p.G; };
    asm volatile("griddepcontrol.wait;" ::: "memory");  // on every path: the call ends after the attention has
    if (T == 0) {
        for (int rho = 8 * grp + warp; rho < rows && rho < 8 * grp + 8; rho += kJoinWarps) {
            const int64_t orow = row_at(rho);
            put(p.out, p.dtype, orow * D + d0 + lane, 0.f);
            put(p.out, p.dtype, orow * D + d0 + 32 + lane, 0.f);
            if (d0 == 0 && lane == 0 && p.lse) p.lse[orow] = -INFINITY;
        }
        return;
    }
    const uint32_t c0 = head_cost(prefix[s], p.pool.Hk) + (uint32_t)h * (T + kHeadCost);
    const int w0 = cut.worker_of(c0 + kHeadCost), w1 = cut.worker_of(c0 + kHeadCost + T - 1);
    if (w0 == w1) return;  // one worker had it all and wrote it
    const int rb = grp / nt, n = grp % nt;
    // the head is its last one for w0 if w0 also has the tile before it
    const int after = c0 > 0 && cut.worker_of(c0 - 1) == w0;
    auto slot_of = [&](int w) { return (((int64_t)rb * p.workers + w) * 2 + (w == w0 ? after : 0)) * nt + n; };
    // row g's largest reference
    float top = -INFINITY;
    for (int w = w0 + t; w <= w1; w += 4) top = fmaxf(top, p.part_rl[slot_of(w) * 8 + g].x);
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float r0 = top == -INFINITY ? 0.f : top;
    float sum = 0.f;  // row g's (the same in the four lanes)
    float4 o[kJoinVecs];
#pragma unroll
    for (int i = 0; i < kJoinVecs; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int wb = w0 + warp; wb <= w1; wb += kJoinWarps * kJoinAtOnce) {
        float2 rl[kJoinAtOnce];
        float4 x[kJoinAtOnce][kJoinVecs];
#pragma unroll
        for (int u = 0; u < kJoinAtOnce; ++u) {
            const int w = wb + u * kJoinWarps;
            const int64_t at = slot_of(w <= w1 ? w : w1);
            rl[u] = p.part_rl[at * 8 + g];
#pragma unroll
            for (int i = 0; i < kJoinVecs; ++i)
                x[u][i] = reinterpret_cast<const float4 *>(p.part_o)[at * (kVec * 32) + (v0 + i) * 32 + lane];
        }
#pragma unroll
        for (int u = 0; u < kJoinAtOnce; ++u) {
            if (wb + u * kJoinWarps > w1) break;
            const float f = exp2f(rl[u].x - r0);
            sum = fmaf(rl[u].y, f, sum);
            const float f0 = __shfl_sync(0xffffffffu, f, 8 * t), f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
            for (int i = 0; i < kJoinVecs; ++i) {
                o[i].x = fmaf(x[u][i].x, f0, o[i].x), o[i].y = fmaf(x[u][i].y, f1, o[i].y);
                o[i].z = fmaf(x[u][i].z, f0, o[i].z), o[i].w = fmaf(x[u][i].w, f1, o[i].w);
            }
        }
    }
    if (t == 0) sums[warp][g] = sum;
    if (warp == 0 && t == 0) refs[g] = r0;
#pragma unroll
    for (int i = 0; i < kJoinVecs; ++i) part[warp][i * 32 + lane] = o[i];
    __syncthreads();
    for (int x = threadIdx.x; x < 8 * 64; x += kJoinWarps * 32) {
        const int row = x >> 6, dim = x & 63, rho = 8 * grp + row;
        if (rho >= rows) continue;
        float total = 0.f, v = 0.f;
#pragma unroll
        for (int k = 0; k < kJoinWarps; ++k) total += sums[k][row];
        // dim 32 b + 16 z + 8 m + g' of row 2 t' + c is component 2 z + c of lane 4 g' + t' of vector 2 b + m
        const int vec = (dim >> 5) * 2 + (dim >> 3 & 1), at = (vec * 32 + (dim & 7) * 4 + (row >> 1)) * 4 + 2 * (dim >> 4 & 1) + (row & 1);
#pragma unroll
        for (int k = 0; k < kJoinWarps; ++k) v += reinterpret_cast<const float *>(part[k])[at];
        const int64_t orow = row_at(rho);
        put(p.out, p.dtype, orow * D + d0 + dim, total == 0.f ? 0.f : v * (1.f / total));
        if (d0 + dim == 0 && p.lse)
            p.lse[orow] = total == 0.f ? -INFINITY : (refs[row] + log2f(total)) * 0.693147180559945309f;
    }
}

// ---------------------------------------------------------------- weights
// w[t] += sum over rows of 2^(score - lse): K tiles only, no join between
// workers (a token is one worker's).  Row passes beyond the first re-read the
// worker's tiles and add to what the first wrote.  Six sequences of 65536 .. 0
// tokens, 4 rows, 24 / 4 heads, D 256, f16: 47 us, 1.9 TB/s of K (90 us in
// passes of 8 rows), bound by latency: 24 rows' query fragments take a warp to
// 255 registers, 8 warps an SM then issue on 40% of the cycles.
struct WeightsParams {
    AttendParams a;
    const float *lse_in;
    const float *prev;
    float *w;
    int64_t width;
    int main_ctas;
};

// Entries no tile covers are prev's (or zero): the CTAs past main_ctas copy
// them, kRest of a (sequence, head) each.
constexpr int kRest = 4096;
__device__ void weights_rest(const WeightsParams &p, int block) {
    const int per = (int)((p.width + kRest - 1) / kRest);
    const int sh = block / per, s = sh / p.a.pool.Hk;
    const int64_t first = ((int64_t)seq_len(p.a.pool, p.a.lens, p.a.table_width, s) + kTile - 1) / kTile * kTile;
    const int64_t from = (int64_t)(block % per) * kRest, row = (int64_t)sh * p.width;
    constexpr int kAtOnce = 8;
    for (int i0 = threadIdx.x; i0 < kRest; i0 += kWarps * 32 * kAtOnce) {
        float v[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int64_t i = from + i0 + u * kWarps * 32;
            v[u] = p.prev && i >= first && i < p.width ? p.prev[row + i] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int64_t i = from + i0 + u * kWarps * 32;
            if (i >= first && i < p.width) p.w[row + i] = v[u];
        }
    }
}

// No accumulators but a tile's scores: more rows fit a pass than in attention.
template <int D, int NT, bool HL>
__host__ __device__ constexpr int weights_ctas_per_sm() {
    return D == 256 ? 2 : (D == 128 ? (NT * (HL ? 2 : 1) >= 4 ? 2 : (NT > 1 || HL ? 3 : 4)) : (NT * (HL ? 2 : 1) >= 4 ? 3 : 4));
}

template <int D, int NT, bool HL>
__global__ void __launch_bounds__(kWarps * 32, weights_ctas_per_sm<D, NT, HL>()) weights_kernel(const WeightsParams wp) {
    constexpr int NST = stages_of<D>(), BYTES = 18 * D;  // the K half of a tile
    const AttendParams &p = wp.a;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[kWarps * NST];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    int2 *prefix = reinterpret_cast<int2 *>(smem + kWarps * NST * BYTES);
    if ((int)blockIdx.x >= wp.main_ctas) {
        weights_rest(wp, (int)blockIdx.x - wp.main_ctas);
        return;
    }
    tile_prefix(p, prefix);
    const Cut cut(prefix, p.n_seq, p.pool.Hk, p.workers);
    const int w = (int)blockIdx.x * kWarps + warp;
    if (w >= (int)cut.W) return;
    const uint32_t u0 = tiles_before(prefix, p.n_seq, p.pool.Hk, cut.begin(w), cut.tiles);
    const uint32_t u1 = tiles_before(prefix, p.n_seq, p.pool.Hk, cut.begin(w + 1), cut.tiles);
    if (u0 >= u1) return;
    const int lg = p.pool.lgP - 5;
    Stages<BYTES, NST> st;
    st.init(smem + warp * NST * BYTES, bars + warp * NST);
    uint32_t phases = 0;
    Query<D, NT, HL> q;
    for (int rho0 = 0; rho0 < p.R * p.G; rho0 += 8 * NT) {
        Cursor<> ahead;
        ahead.seek(p, prefix, u0, lg);
        Place at = ahead;
        const int units = (int)(u1 - u0);
        int fetched = 0;
#pragma unroll
        for (int i = 0; i < NST; ++i) {
            if (fetched < units) {
                st.fetch(i, ahead.tile(p, lg, 36 * D));
                ahead.advance(p, prefix, lg);
                ++fetched;
            }
        }
        bool fresh = true;
        int stage = 0, unit = 0;
        if (p.give_up) st.give_up(stage, phases);
        float2 lse2[NT], fac[NT];  // rows 2t, 2t + 1
        int len = 0;
        for (; unit < units; ++unit) {
            if (fresh) {
                typename Query<D, NT, HL>::Raw raw;
                raw.load(p, at.s, at.h, rho0);
                len = seq_len(p.pool, p.lens, p.table_width, at.s);
                q.form(p, raw, rho0);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int rho = rho0 + 8 * n + g;
                    float z = INFINITY;  // rows past the last, and rows that saw nothing, add nothing
                    if (rho < p.R * p.G) {
                        z = wp.lse_in[((int64_t)at.s * p.R + rho / p.G) * p.Hq + at.h * p.G + rho % p.G] * 1.4426950408889634f;
                        if (z == -INFINITY) z = INFINITY;
                    }
                    lse2[n] = make_float2(__shfl_sync(0xffffffffu, z, 8 * t), __shfl_sync(0xffffffffu, z, 8 * t + 4));
                    fac[n] = make_float2(__shfl_sync(0xffffffffu, q.fac[n], 8 * t), __shfl_sync(0xffffffffu, q.fac[n], 8 * t + 4));
                }
                fresh = false;
            }
            const int in_tile = len - at.k * kTile;
            float sum[4];  // tokens g, g + 8, g + 16, g + 24
            if (!st.wait(stage, phases)) {
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[i] = __int_as_float(0x7fc00000);
                if (st.gave_up) break;
            } else {
                float acc[2][NT][4];
#pragma unroll
                for (int c = 0; c < 2; ++c) q.scores(st.buf + stage * BYTES, c, acc[c]);
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[i] = 0.f;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int base = in_tile - (p.R - 1), rho = rho0 + 8 * n + 2 * t;
                    const int see0 = base + rho / p.G, see1 = base + (rho + 1) / p.G;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float *a = &acc[i >> 1][n][2 * (i & 1)];
                        const float e0 = ex2(fmaf(a[0], fac[n].x, -lse2[n].x)), e1 = ex2(fmaf(a[1], fac[n].y, -lse2[n].y));
                        sum[i] += (8 * i + g < see0 ? e0 : 0.f) + (8 * i + g < see1 ? e1 : 0.f);
                    }
                }
            }
            // over the row pairs t: each exchange halves the values a lane keeps
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float give = (t & 2) ? sum[i] : sum[i + 2], keep = (t & 2) ? sum[i + 2] : sum[i];
                sum[i] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
            }
            {
                const float give = (t & 1) ? sum[0] : sum[1], keep = (t & 1) ? sum[1] : sum[0];
                sum[0] = keep + __shfl_xor_sync(0xffffffffu, give, 1);
            }
            const int tok = 8 * t + g;
            const int64_t pos = (int64_t)at.k * kTile + tok;
            if (pos < wp.width) {
                const int64_t o = ((int64_t)at.s * p.pool.Hk + at.h) * wp.width + pos;
                const float before = rho0 ? wp.w[o] : (wp.prev ? wp.prev[o] : 0.f);
                wp.w[o] = before + (tok < in_tile ? sum[0] : 0.f);
            }
            __syncwarp();
            if (fetched < units) {
                st.fetch(stage, ahead.tile(p, lg, 36 * D));
                ahead.advance(p, prefix, lg);
                ++fetched;
            }
            if (at.k + 1 == at.T) fresh = true;
            stage = stage + 1 == NST ? 0 : stage + 1;
            at.next(prefix, p.n_seq, p.pool.Hk);
        }
        if (st.gave_up) {  // every token of this worker's range is NaN, the entries past a sequence's length are prev's
            st.drain(stage, fetched - unit, phases);
            Cursor<> c;
            c.seek(p, prefix, u0, lg);
            for (int x = 0; x < units; ++x) {
                const int64_t pos = (int64_t)c.k * kTile + lane, o = ((int64_t)c.s * p.pool.Hk + c.h) * wp.width + pos;
                if (pos < wp.width)
                    wp.w[o] = pos < seq_len(p.pool, p.lens, p.table_width, c.s) ? __int_as_float(0x7fc00000) : wp.prev ? wp.prev[o] : 0.f;
                c.next(prefix, p.n_seq, p.pool.Hk);
            }
            return;
        }
    }
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
size_t elem_size(int dtype) { return dtype == KVS_F32 ? 4 : 2; }

bool dtype_ok(int32_t t) { return t == KVS_F32 || t == KVS_F16 || t == KVS_BF16; }

// How a call's query rows are passed: fp32 queries 8 rows at a time (with
// their lo halves), 16-bit ones 8 if that is all there are, else 16.  At
// D = 256 the 16-row accumulators do not fit the registers.
struct Shape {
    int nt, row_blocks, workers, ctas;
    bool hl;
};
Shape shape_of(uint32_t D, uint32_t rows, int32_t dtype, int sms) {
    Shape s;
    s.hl = dtype == KVS_F32;
    s.nt = (!s.hl && D <= 128 && rows > 8) ? 2 : 1;
    s.row_blocks = ((int)rows + 8 * s.nt - 1) / (8 * s.nt);
    int ranges = sms * attend_ctas((int)D, s.nt) / s.row_blocks;
    if (ranges < 1) ranges = 1;
    s.ctas = ranges * s.row_blocks;
    s.workers = ranges * kWarps;
    return s;
}
constexpr int kSmsAssumed = 152;  // sizes the workspace; a launch uses no more than that many SMs' worth

uint64_t workspace_of(const Shape &s, uint32_t D) {
    const uint64_t rows = (uint64_t)s.row_blocks * s.workers * 2 * 8 * s.nt;
    return (rows * D * 4 + rows * 8 + 255) / 256 * 256;
}

kvs_status check_rows(uint32_t n_seq, uint32_t n_rows, uint32_t n_q_head, int Hk, uint32_t *group) {
    if (n_seq > kMaxSeq) return bad(KVS_ERR_UNSUPPORTED, "n_seq must be at most 4096");
    if (n_rows < 1 || n_q_head < (uint32_t)Hk || n_q_head % (uint32_t)Hk != 0)
        return bad(KVS_ERR_INVALID, "need n_rows >= 1 and n_q_head a positive multiple of n_kv_head");
    *group = n_q_head / (uint32_t)Hk;
    if (*group > (uint32_t)kMaxGroupRows || n_rows > (uint32_t)kMaxGroupRows || *group * n_rows > (uint32_t)kMaxGroupRows)
        return bad(KVS_ERR_UNSUPPORTED, "n_rows * (n_q_head / n_kv_head) must be <= 64");
    return KVS_OK;
}

kvs_status fill_attend(const kvs_q4_pool *pool, const int32_t *table, uint32_t table_width, const int32_t *lens, uint32_t n_seq,
                       uint32_t n_rows, uint32_t n_q_head, const void *q, int32_t dtype, uint64_t q_stride, float scale,
                       AttendParams *p) {
    kvs_status s = check_q4_pool(pool, true, &p->pool);
    if (s != KVS_OK) return s;
    if (!dtype_ok(dtype)) return bad(KVS_ERR_INVALID, "dtype must be KVS_F32, KVS_F16 or KVS_BF16");
    uint32_t G = 0;
    s = check_rows(n_seq, n_rows, n_q_head, p->pool.Hk, &G);
    if (s != KVS_OK) return s;
    if (n_seq && (!table || !lens || !q)) return bad(KVS_ERR_INVALID, "null table, lens or q");
    if (table_width < 1 || (uint64_t)table_width * pool->page_tokens > 0x7fffffc0ull)
        return bad(KVS_ERR_INVALID, "table_width * page_tokens must be 1 .. 2^31 - 64");
    const uint64_t line = (uint64_t)n_seq * pool->n_kv_head * ((uint64_t)table_width * (pool->page_tokens / 32) + kHeadCost);
    if (line > 0x7fffffffull) return bad(KVS_ERR_UNSUPPORTED, "n_seq * n_kv_head * (table_width * page_tokens / 32 + 6) must be below 2^31");
    if (!aligned(q, 16) || (q_stride * elem_size(dtype)) % 16 != 0 || q_stride < (uint64_t)n_q_head * pool->head_dim)
        return bad(KVS_ERR_INVALID, "q rows must start on 16-byte boundaries, at least n_q_head * head_dim apart");
    if (!isfinite(scale)) return bad(KVS_ERR_INVALID, "scale must be finite");
    p->table = table;
    p->table_width = (int)table_width;
    p->lens = lens;
    p->n_seq = (int)n_seq;
    p->R = (int)n_rows;
    p->Hq = (int)n_q_head;
    p->G = (int)G;
    p->q = q;
    p->dtype = dtype;
    p->q_stride = (int64_t)q_stride;
    p->scale_log2 = scale * 1.4426950408889634f;
    return KVS_OK;
}

template <typename P, typename... A>
cudaError_t launch(void (*kernel)(P, A...), dim3 grid, int threads, int smem, cudaStream_t s, bool pdl, const P &p, A... a) {
    // The 48 KB that need no opt-in are of dynamic and static bytes together: 256 static ones in the attention and the
    // weights, 9 KB in the join by 4 warps, 33 KB in the one by 16, whose dynamic ones are those of fewer sequences than SMs.
    // (Below, the look-up is left out: 0.3 us.)
    if (smem > 36 * 1024) {
        const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(kernel), smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p, a...);
}

int smem_of(uint32_t D, int bytes, int turn, uint32_t n_seq) {
    return kWarps * ((D == 64 ? 4 : 3) * bytes + turn) + ((int)n_seq + 1) * 8;
}

}  // namespace

kvs_status check_q4_pool(const kvs_q4_pool *pool, bool need_pages, Q4Pool *out) {
    if (!pool) return bad(KVS_ERR_INVALID, "null pool");
    const uint32_t P = pool->page_tokens, D = pool->head_dim;
    if (!(P == 32 || P == 64 || P == 128 || P == 256) || !(D == 64 || D == 128 || D == 256))
        return bad(KVS_ERR_UNSUPPORTED, "page_tokens must be 32..256 (power of two), head_dim 64, 128 or 256");
    if (pool->n_kv_head == 0 || pool->n_kv_head > 65535) return bad(KVS_ERR_INVALID, "n_kv_head must be 1 .. 65535");
    if (need_pages) {
        if (!pool->pages || !aligned(pool->pages, 16)) return bad(KVS_ERR_INVALID, "pages null or not 16-byte aligned");
        if (pool->n_pages == 0 || pool->n_pages > 0x7fffffffull) return bad(KVS_ERR_INVALID, "n_pages must be 1 .. 2^31 - 1");
    }
    out->pages = static_cast<uint8_t *>(pool->pages);
    out->n_pages = (int64_t)pool->n_pages;
    out->P = (int)P;
    out->lgP = P == 32 ? 5 : P == 64 ? 6 : P == 128 ? 7 : 8;
    out->Hk = (int)pool->n_kv_head;
    out->head_bytes = (int64_t)P * D * 9 / 8;
    out->page_bytes = out->head_bytes * out->Hk;
    return KVS_OK;
}

}  // namespace kvs

using namespace kvs;

extern "C" kvs_status kvs_q4_query_sizes(const kvs_q4_pool *pool, uint32_t n_rows, uint32_t n_q_head, int32_t dtype,
                                         uint64_t *page_bytes, uint64_t *workspace_bytes) {
    Pool p = {};
    kvs_status s = check_q4_pool(pool, false, &p);
    if (s != KVS_OK) return s;
    if (workspace_bytes) {
        if (!dtype_ok(dtype)) return bad(KVS_ERR_INVALID, "dtype must be KVS_F32, KVS_F16 or KVS_BF16");
        uint32_t G = 0;
        s = check_rows(1, n_rows, n_q_head, p.Hk, &G);
        if (s != KVS_OK) return s;
        *workspace_bytes = workspace_of(shape_of(pool->head_dim, n_rows * G, dtype, kSmsAssumed), pool->head_dim);
    }
    if (page_bytes) *page_bytes = (uint64_t)p.page_bytes;
    return KVS_OK;
}

static kvs_status rows_call(const kvs_q4_pool *pool, const int64_t *slots, uint64_t n, int32_t dtype, RowsParams *p) {
    kvs_status s = check_q4_pool(pool, true, &p->pool);
    if (s != KVS_OK) return s;
    if (!dtype_ok(dtype)) return bad(KVS_ERR_INVALID, "dtype must be KVS_F32, KVS_F16 or KVS_BF16");
    if (n && (!slots || !aligned(slots, 8))) return bad(KVS_ERR_INVALID, "slots null or misaligned");
    const uint64_t units = (uint64_t)pool->n_kv_head * (pool->head_dim / 32);
    // (so that the launch's CTAs, 256 of K's and V's blocks each or 32 V rows of a head, stay below 2^31)
    if (n > (1ull << 36) / units) return bad(KVS_ERR_INVALID, "too many rows");
    p->slots = slots;
    p->n = (int64_t)n;
    p->dtype = dtype;
    return KVS_OK;
}

extern "C" kvs_status kvs_q4_append(const kvs_q4_pool *pool, const int64_t *slots, uint64_t n, const void *k, const void *v,
                                    int32_t dtype, uint64_t k_stride, uint64_t v_stride, void *stream) {
    RowsParams p = {};
    kvs_status s = rows_call(pool, slots, n, dtype, &p);
    if (s != KVS_OK) return s;
    if (n == 0) return KVS_OK;
    const uint64_t row = (uint64_t)pool->n_kv_head * pool->head_dim, e = elem_size(dtype);
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || k_stride < row || v_stride < row || k_stride * e % 16 || v_stride * e % 16)
        return bad(KVS_ERR_INVALID, "k and v rows must start on 16-byte boundaries, at least n_kv_head * head_dim apart");
    p.k = k;
    p.v = v;
    p.k_stride = (int64_t)k_stride;
    p.v_stride = (int64_t)v_stride;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const uint32_t D = pool->head_dim;
    const uint64_t blocks = (n * (row / 32) + 64 * kInFlight - 1) / (64 * kInFlight);
    const uint64_t v_blocks = (n + 31) / 32 * pool->n_kv_head;
    auto kernel = D == 64 ? append_kernel<64, false> : D == 128 ? append_kernel<128, false> : append_kernel<256, false>;
    if (dtype == KVS_F32) kernel = D == 64 ? append_kernel<64, true> : D == 128 ? append_kernel<128, true> : append_kernel<256, true>;
    const cudaError_t ce = launch(kernel, dim3((unsigned)(blocks + v_blocks)), 256, 0, st, false, p, (int)blocks);
    return ce == cudaSuccess ? KVS_OK : cuda_failed("append launch", ce);
}

extern "C" kvs_status kvs_q4_read(const kvs_q4_pool *pool, const int64_t *slots, uint64_t n, void *k, void *v, int32_t dtype,
                                  void *stream) {
    RowsParams p = {};
    kvs_status s = rows_call(pool, slots, n, dtype, &p);
    if (s != KVS_OK) return s;
    if (!aligned(k, 16) || !aligned(v, 16)) return bad(KVS_ERR_INVALID, "k and v must be 16-byte aligned");
    if (n == 0 || (!k && !v)) return KVS_OK;
    p.ko = k;
    p.vo = v;
    const uint64_t pairs = n * pool->n_kv_head * (pool->head_dim / 64);
    auto kernel = pool->head_dim == 64 ? read_kernel<64> : pool->head_dim == 128 ? read_kernel<128> : read_kernel<256>;
    const cudaError_t ce = launch(kernel, dim3((unsigned)((pairs + 64 * kPairs - 1) / (64 * kPairs)), 2), 256, 0, static_cast<cudaStream_t>(stream), false, p);
    return ce == cudaSuccess ? KVS_OK : cuda_failed("read launch", ce);
}

template <bool WIN>
static kvs_status attend_call(const kvs_q4_pool *pool, AttendParams &p, void *out, float *lse, void *workspace, uint64_t workspace_bytes,
                              void *stream) {
    const uint32_t D = pool->head_dim, n_seq = (uint32_t)p.n_seq, n_rows = (uint32_t)p.R;
    const int32_t dtype = p.dtype;
    const uint64_t need = workspace_of(shape_of(D, n_rows * p.G, dtype, kSmsAssumed), D);
    if (!workspace || !aligned(workspace, 256)) return bad(KVS_ERR_INVALID, "workspace null or not 256-byte aligned");
    if (workspace_bytes < need) return bad(KVS_ERR_CAPACITY, "workspace smaller than kvs_q4_query_sizes asks for");
    const int sms = current_device_sms();
    const Shape sh = shape_of(D, n_rows * p.G, dtype, sms < kSmsAssumed ? sms : kSmsAssumed);
    p.give_up = batch_fault() == KVS_FAULT_DEVICE_WAIT;
    p.out = out;
    p.lse = lse;
    p.row_blocks = sh.row_blocks;
    p.workers = sh.workers;
    p.part_o = static_cast<float *>(workspace);
    p.part_rl = reinterpret_cast<float2 *>(p.part_o + (uint64_t)sh.row_blocks * sh.workers * 2 * 8 * sh.nt * D);
    void (*k)(AttendParams) = nullptr;
    if (D == 64) k = sh.hl ? attend_kernel<64, 1, true, WIN> : sh.nt == 2 ? attend_kernel<64, 2, false, WIN> : attend_kernel<64, 1, false, WIN>;
    if (D == 128) k = sh.hl ? attend_kernel<128, 1, true, WIN> : sh.nt == 2 ? attend_kernel<128, 2, false, WIN> : attend_kernel<128, 1, false, WIN>;
    if (D == 256) k = sh.hl ? attend_kernel<256, 1, true, WIN> : attend_kernel<256, 1, false, WIN>;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = launch(k, dim3(sh.ctas), kWarps * 32, smem_of(D, 36 * (int)D, turn_bytes((int)D, sh.nt), n_seq), st, false, p);
    if (e != cudaSuccess) return cuda_failed("attention launch", e);
    // 16 warps where few CTAs join many partials each (one sequence of 4096 tokens: 13.8 us with its attention, 15.4 with 4
    // warps), 4 in a batch, where a head has a handful of them (32 sequences: 90.8 us, 96.7 with 16)
    const uint64_t groups = (uint64_t)n_seq * pool->n_kv_head * ((n_rows * p.G + 7) / 8);
    const bool few = groups * (D / 64) < (uint64_t)sms;
    void (*c)(AttendParams, int) = few ? (D == 64 ? combine_kernel<64, 16, WIN> : D == 128 ? combine_kernel<128, 16, WIN> : combine_kernel<256, 16, WIN>)
                                       : (D == 64 ? combine_kernel<64, 4, WIN> : D == 128 ? combine_kernel<128, 4, WIN> : combine_kernel<256, 4, WIN>);
    e = launch(c, dim3((unsigned)groups, D / 64), few ? 512 : 128, ((int)n_seq + 1) * 8, st, true, p, sh.nt);
    return e == cudaSuccess ? KVS_OK : cuda_failed("combine launch", e);
}

extern "C" kvs_status kvs_q4_attend(const kvs_q4_pool *pool, const int32_t *table, uint32_t table_width, const int32_t *lens,
                                    uint32_t n_seq, uint32_t n_rows, uint32_t n_q_head, const void *q, int32_t dtype,
                                    uint64_t q_stride, float scale, void *out, float *lse, void *workspace,
                                    uint64_t workspace_bytes, void *stream) {
    AttendParams p = {};
    kvs_status s = fill_attend(pool, table, table_width, lens, n_seq, n_rows, n_q_head, q, dtype, q_stride, scale, &p);
    if (s != KVS_OK) return s;
    if (n_seq == 0) return KVS_OK;
    if (!out || !aligned(out, 16)) return bad(KVS_ERR_INVALID, "out null or not 16-byte aligned");
    return attend_call<false>(pool, p, out, lse, workspace, workspace_bytes, stream);
}

extern "C" kvs_status kvs_q4_attend_window(const kvs_q4_pool *pool, const int32_t *table, uint32_t table_width, const int32_t *lens,
                                           uint32_t n_seq, uint32_t n_rows, uint32_t n_q_head, const void *q, int32_t dtype,
                                           uint64_t q_stride, float scale, uint32_t window, uint32_t sinks, void *out, float *lse,
                                           void *workspace, uint64_t workspace_bytes, void *stream) {
    AttendParams p = {};
    kvs_status s = fill_attend(pool, table, table_width, lens, n_seq, n_rows, n_q_head, q, dtype, q_stride, scale, &p);
    if (s != KVS_OK) return s;
    if (window > 0x7fffffffu || sinks > 0x7fffffffu - 64u) return bad(KVS_ERR_INVALID, "window must be at most 2^31 - 1, sinks 2^31 - 65");
    if (n_seq == 0) return KVS_OK;
    if (!out || !aligned(out, 16)) return bad(KVS_ERR_INVALID, "out null or not 16-byte aligned");
    if (window == 0 || window >= (uint64_t)table_width * pool->page_tokens)  // every token is inside
        return attend_call<false>(pool, p, out, lse, workspace, workspace_bytes, stream);
    p.window = (int)window;
    p.sinks = (int)sinks;
    return attend_call<true>(pool, p, out, lse, workspace, workspace_bytes, stream);
}

extern "C" kvs_status kvs_q4_weights(const kvs_q4_pool *pool, const int32_t *table, uint32_t table_width, const int32_t *lens,
                                     uint32_t n_seq, uint32_t n_rows, uint32_t n_q_head, const void *q, int32_t dtype,
                                     uint64_t q_stride, float scale, const float *lse, const float *prev, float *weights,
                                     uint64_t width, void *stream) {
    WeightsParams p = {};
    kvs_status s = fill_attend(pool, table, table_width, lens, n_seq, n_rows, n_q_head, q, dtype, q_stride, scale, &p.a);
    if (s != KVS_OK) return s;
    if (n_seq && width && (!lse || !weights)) return bad(KVS_ERR_INVALID, "null lse or weights");
    if (width > 0x7fffffffull) return bad(KVS_ERR_INVALID, "width must be at most 2^31 - 1");
    if (n_seq == 0 || width == 0) return KVS_OK;
    p.a.give_up = batch_fault() == KVS_FAULT_DEVICE_WAIT;
    const uint32_t D = pool->head_dim, rows = n_rows * p.a.G;
    const bool hl = dtype == KVS_F32;
    // up to 16 or (16-bit queries) 32 rows a pass: the fewer passes, the fewer times a tile is read; the passes as even as
    // eights of rows allow (24 rows of six sequences of 65536 .. 0 tokens: 47 us, 52 as 32)
    const int eights = (int)(rows + 7) / 8, most = hl ? 2 : 4, passes = (eights + most - 1) / most;
    const int nt = (eights + passes - 1) / passes;
    void (*k)(WeightsParams) = nullptr;
    int per_sm = 0;
#define KVS_PICK(d, n, h)                 \
    if (D == d && nt == n && hl == h) {   \
        k = weights_kernel<d, n, h>;      \
        per_sm = weights_ctas_per_sm<d, n, h>(); \
    }
    KVS_PICK(64, 1, false) KVS_PICK(64, 2, false) KVS_PICK(64, 3, false) KVS_PICK(64, 4, false) KVS_PICK(64, 1, true) KVS_PICK(64, 2, true)
    KVS_PICK(128, 1, false) KVS_PICK(128, 2, false) KVS_PICK(128, 3, false) KVS_PICK(128, 4, false) KVS_PICK(128, 1, true) KVS_PICK(128, 2, true)
    KVS_PICK(256, 1, false) KVS_PICK(256, 2, false) KVS_PICK(256, 3, false) KVS_PICK(256, 4, false) KVS_PICK(256, 1, true) KVS_PICK(256, 2, true)
#undef KVS_PICK
    p.main_ctas = current_device_sms() * per_sm;
    p.a.row_blocks = 1;
    p.a.workers = p.main_ctas * kWarps;
    p.lse_in = lse;
    p.prev = prev;
    p.w = weights;
    p.width = (int64_t)width;
    const uint64_t rest = prev != weights ? (uint64_t)n_seq * pool->n_kv_head * ((width + kRest - 1) / kRest) : 0;
    if (rest > 0x7fffffffull - (uint64_t)p.main_ctas) return bad(KVS_ERR_UNSUPPORTED, "n_seq * n_kv_head * width too large for one launch");
    const cudaError_t e = launch(k, dim3((unsigned)(p.main_ctas + rest)), kWarps * 32, smem_of(D, 18 * (int)D, 0, n_seq),
                                 static_cast<cudaStream_t>(stream), false, p);
    return e == cudaSuccess ? KVS_OK : cuda_failed("weights launch", e);
}
