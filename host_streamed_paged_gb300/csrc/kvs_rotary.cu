// Rotary positions of query and key rows, with or without a norm of every head
// before them (include/kvs.h, kvs_rotate and kvs_norm_rotate).
//
// Angles.  A pair's angle at position p is p f.  Kept as turns in 64-bit fixed
// point (f / 2 pi times 2^64), p times it modulo 2^64 is the angle's fraction of
// a turn, exact but for p times the last bit's rounding; its top 32 bits, read as signed, are
// the angle in half turns, -1 .. 1, for sincospif.  (p f in fp32 is off by p f
// 2^-24: 0.06 radians at a million.)
//
// Bound by bytes: every element once in, once out.  A lane holds 16 elements of
// a head, both sides of its 8 pairs, so a pair never crosses lanes and a row may
// be its own output; D / 16 lanes share a head, and the 512 / D heads that a
// warp takes at a time share the work of the row's angles.
//
// A warp's job is as many of a row's steps (512 elements) as leave the card's
// warp slots one job each, a whole row from some 5000 rows on: the angles, 8
// sincospif a lane at most, are formed once a job and the next step's elements
// are on their way meanwhile.  The arithmetic is in paired fp32 instructions
// (3000 rows with norms 13.2 -> 11.8 us).
//
// Measured: 16755 rows of 24 + 4 heads, D 256, 64 dims rotated, f16: 75.2 us, 6.4
// TB/s (94% of a copy's rate; ncu: DRAM 73% of its peak).  With norms, 12001
// rows of 32 + 8 heads, D 128, bf16: 49.2 us, 5.0 TB/s: 54% of the issue slots
// taken at 80 registers, so the loads in flight and the instructions bound it
// together.  (Two steps on their way instead of one: 55.7 us, fewer warps fit; 28
// warps an SM at 72 registers: 46.6, but f16 51.7 against 49.6 and fp32 92
// against 76.)  A step of 64 rows takes 2.1 us of the GPU, 16 with the call.
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

constexpr int kThreads = 128;

struct Side {
    const void *x;
    void *y;
    int64_t x_stride, y_stride;
    int heads, steps;  // steps: of a warp, 512 / D heads each
    const void *weight;
};

struct RotaryParams {
    const uint64_t *turns;
    const void *pos;
    int wide_pos;  // int64 positions
    int64_t n;
    int rot, interleaved;
    float magnitude;
    Side side[2];
    int per, jobs;  // steps of a warp's job, jobs of a row
    int weight_type;
    float eps;
};

using tc::fma2;
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(*reinterpret_cast<uint64_t *>(&r))
        : "l"(*reinterpret_cast<const uint64_t *>(&a)), "l"(*reinterpret_cast<const uint64_t *>(&b)));
    return r;
}
__device__ __forceinline__ float2 two(uint32_t w, bool bf16) {
    if (bf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// 8 consecutive elements, as they lie in memory
template <int DT>
struct Eight {
    uint4 w[DT == KVS_F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        const uint4 *at = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p) + i * (DT == KVS_F32 ? 4 : 2));
        w[0] = at[0];
        if constexpr (DT == KVS_F32) w[1] = at[1];
    }
    __device__ __forceinline__ void get(float *x) const {
        if constexpr (DT == KVS_F32) {
            x[0] = __uint_as_float(w[0].x), x[1] = __uint_as_float(w[0].y), x[2] = __uint_as_float(w[0].z), x[3] = __uint_as_float(w[0].w);
            x[4] = __uint_as_float(w[1].x), x[5] = __uint_as_float(w[1].y), x[6] = __uint_as_float(w[1].z), x[7] = __uint_as_float(w[1].w);
        } else {
            const float2 a = two(w[0].x, DT == KVS_BF16), b = two(w[0].y, DT == KVS_BF16), c = two(w[0].z, DT == KVS_BF16), d = two(w[0].w, DT == KVS_BF16);
            x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y, x[4] = c.x, x[5] = c.y, x[6] = d.x, x[7] = d.y;
        }
    }
    static __device__ __forceinline__ void store(void *p, int64_t i, const float *x) {
        if constexpr (DT == KVS_F32) {
            float4 *at = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
            at[0] = make_float4(x[0], x[1], x[2], x[3]);
            at[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (DT == KVS_BF16) {
                    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
                    o[k] = *reinterpret_cast<const uint32_t *>(&v);
                } else {
                    const __half2 v = __floats2half2_rn(x[2 * k], x[2 * k + 1]);
                    o[k] = *reinterpret_cast<const uint32_t *>(&v);
                }
            }
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
};

template <int D, int DT, bool NORM>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
    constexpr int L = D / 16, HS = 32 / L, EACH = 8 / HS;  // lanes of a head, heads of a step, pairs whose angles a lane forms
    const int lane = threadIdx.x & 31, l = lane % L, slot = lane / L;
    const int64_t job = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t row = job / p.jobs;
    if (row >= p.n) return;
    const int first = (int)(job - row * p.jobs) * p.per, steps = p.side[0].steps + p.side[1].steps;
    const int last = first + p.per < steps ? first + p.per : steps;
    // the lane's dims: 8 from a, 8 from b.  Pairs of halves: (a + j, b + j) are pair 8 l + j; of neighbours: a .. b + 7 is one
    // run of 16 dims.  Lanes past the rotated part copy such runs.
    const bool turned = 16 * l < p.rot;
    const int a = p.interleaved || !turned ? 16 * l : 8 * l, b = p.interleaved || !turned ? a + 8 : p.rot / 2 + 8 * l;

    struct Data {
        Eight<DT> a, b;
    };
    auto load = [&](int step, Data &d) {  // false: no head of this lane
        const Side &s = p.side[step >= p.side[0].steps];
        const int h = (step >= p.side[0].steps ? step - p.side[0].steps : step) * HS + slot;
        if (h >= s.heads) return false;
        const int64_t at = row * s.x_stride + (int64_t)h * D;
        d.a.load(s.x, at + a);
        d.b.load(s.x, at + b);
        return true;
    };
    Data next;
    bool have = load(first, next);

    float c[8], s[8];
    {
        const int64_t at = p.wide_pos ? static_cast<const int64_t *>(p.pos)[row] : static_cast<const int32_t *>(p.pos)[row];
        float ce[EACH], se[EACH];
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
            const int pair = 8 * l + slot * EACH + k;
            const uint64_t t = turned ? p.turns[pair] : 0;
            const int32_t half_turns = (int32_t)((uint64_t)at * t >> 32);
            sincospif((float)half_turns * 4.6566128730773926e-10f, &se[k], &ce[k]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            c[j] = __shfl_sync(0xffffffffu, ce[j % EACH], j / EACH * L + l) * p.magnitude;
            s[j] = __shfl_sync(0xffffffffu, se[j % EACH], j / EACH * L + l) * p.magnitude;
        }
    }
    float w[NORM ? 16 : 1];
    int weighted = -1;  // the side that w is of
    for (int step = first; step < last; ++step) {
        const Data now = next;
        const bool mine = have;
        if (step + 1 < last) have = load(step + 1, next);
        const int which = step >= p.side[0].steps;
        const Side &sd = p.side[which];
        float x[16];
        now.a.get(x);
        now.b.get(x + 8);
        if constexpr (NORM) {
            if (weighted != which) {
                weighted = which;
#pragma unroll
                for (int j = 0; j < 16; ++j) w[j] = 1.f;
                if (sd.weight) {
                    auto take = [&](auto t) {
                        Eight<decltype(t)::value> v;
                        v.load(sd.weight, a);
                        v.get(w);
                        v.load(sd.weight, b);
                        v.get(w + 8);
                    };
                    if (p.weight_type == KVS_F32) take(std::integral_constant<int, KVS_F32>{});
                    else if (p.weight_type == KVS_F16) take(std::integral_constant<int, KVS_F16>{});
                    else take(std::integral_constant<int, KVS_BF16>{});
                }
            }
            if (!mine) {
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = 1.f;
            }
            auto over_head = [&](float sum) {
#pragma unroll
                for (int o = 1; o < L; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                return sum * (1.f / D);
            };
            float2 *x2 = reinterpret_cast<float2 *>(x), square = mul2(x2[0], x2[0]);
#pragma unroll
            for (int j = 1; j < 8; ++j) square = fma2(x2[j], x2[j], square);
            const float v = over_head(square.x + square.y) + p.eps;
            float inv = rsqrtf(v);
            inv = fmaf(inv * 0.5f, fmaf(-v * inv, inv, 1.f), inv);  // (one step of Newton's)
            const bool odd = !(v >= 7.9e-31f && v <= 1.3e36f);  // squares near or past fp32's ends: 2^-100, 2^120
            if (__any_sync(0xffffffffu, odd)) {
                // again with the larger of the head's largest element and eps's root brought to 1 .. 2
                float top = sqrtf(p.eps);
#pragma unroll
                for (int j = 0; j < 16; ++j) top = fmaxf(top, fabsf(x[j]));
#pragma unroll
                for (int o = 1; o < L; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                int e = (int)(__float_as_uint(top) >> 23) - 127;
                e = e < -120 ? -120 : (e > 120 ? 120 : e);
                const float f = __uint_as_float((uint32_t)(127 - e) << 23);
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 16; ++j) sum = fmaf(x[j] * f, x[j] * f, sum);
                const float root = __frsqrt_rn(over_head(sum) + p.eps * f * f);
                // (elements are brought up before the root's product: root f passes fp32 where they are subnormal.  Down, f
                // goes with the root: small elements beside a large one keep their bits)
                if (odd) {
                    const float up = fmaxf(f, 1.f);
                    inv = root * fminf(f, 1.f);
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[j] *= up;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) x2[j] = mul2(mul2(x2[j], make_float2(inv, inv)), make_float2(w[2 * j], w[2 * j + 1]));
        }
        if (!mine) continue;
        if (turned) {
            if (p.interleaved) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float u = x[2 * j], v = x[2 * j + 1];
                    x[2 * j] = u * c[j] - v * s[j];
                    x[2 * j + 1] = v * c[j] + u * s[j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float2 u = make_float2(x[j], x[j + 1]), v = make_float2(x[8 + j], x[9 + j]);
                    const float2 c2 = make_float2(c[j], c[j + 1]), s2 = make_float2(s[j], s[j + 1]), n2 = make_float2(-s[j], -s[j + 1]);
                    const float2 a2 = fma2(v, n2, mul2(u, c2)), b2 = fma2(u, s2, mul2(v, c2));
                    x[j] = a2.x, x[j + 1] = a2.y, x[8 + j] = b2.x, x[9 + j] = b2.y;
                }
            }
        }
        const int h = (which ? step - p.side[0].steps : step) * HS + slot;
        const int64_t at = row * sd.y_stride + (int64_t)h * D;
        Eight<DT>::store(sd.y, at + a, x);
        Eight<DT>::store(sd.y, at + b, x + 8);
    }
}

// ---------------------------------------------------------------- host side

kvs_status bad(kvs_status s, const char *why) {
    set_thread_error(why);
    return s;
}
bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool type_ok(int32_t t) { return t == KVS_F32 || t == KVS_F16 || t == KVS_BF16; }

template <int D, bool NORM>
auto kernel_for(int32_t dtype) {
    return dtype == KVS_F32 ? rotary_kernel<D, KVS_F32, NORM> : dtype == KVS_F16 ? rotary_kernel<D, KVS_F16, NORM> : rotary_kernel<D, KVS_BF16, NORM>;
}

kvs_status rotary_call(const kvs_rotary *r, const void *positions, uint32_t position_bytes, uint64_t n, int32_t dtype,
                       const kvs_head_rows *q, const kvs_head_rows *k, bool norm, int32_t weight_dtype, float eps, void *stream) {
    if (!r || !q) return bad(KVS_ERR_INVALID, "null rotary or q");
    const uint32_t D = r->head_dim;
    if (!(D == 64 || D == 128 || D == 256)) return bad(KVS_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
    if (r->rot_dim > D || r->rot_dim % 16) return bad(KVS_ERR_UNSUPPORTED, "rot_dim must be a multiple of 16, at most head_dim");
    if (r->rot_dim && (!r->turns || !aligned(r->turns, 8))) return bad(KVS_ERR_INVALID, "turns null or misaligned");
    if (!isfinite(r->magnitude)) return bad(KVS_ERR_INVALID, "magnitude must be finite");
    if (!type_ok(dtype)) return bad(KVS_ERR_INVALID, "dtype must be KVS_F32, KVS_F16 or KVS_BF16");
    if (position_bytes != 4 && position_bytes != 8) return bad(KVS_ERR_INVALID, "positions are of 4 or 8 bytes");
    if (norm && !type_ok(weight_dtype)) return bad(KVS_ERR_INVALID, "weight_dtype must be KVS_F32, KVS_F16 or KVS_BF16");
    if (norm && !(eps >= 0.f && isfinite(eps))) return bad(KVS_ERR_INVALID, "eps must be finite and not negative");
    RotaryParams p = {};
    const uint64_t size = dtype == KVS_F32 ? 4 : 2, heads_a_step = 512 / D;
    for (int i = 0; i < 2; ++i) {
        const kvs_head_rows *x = i ? k : q;
        if (!x) continue;
        if (x->n_head == 0 || x->n_head > 65535) return bad(KVS_ERR_INVALID, "n_head must be 1 .. 65535");
        const uint64_t row = (uint64_t)x->n_head * D;
        if (n && (!x->x || !x->y || !aligned(x->x, 16) || !aligned(x->y, 16))) return bad(KVS_ERR_INVALID, "rows null or not 16-byte aligned");
        if (x->x_stride < row || x->y_stride < row || x->x_stride * size % 16 || x->y_stride * size % 16)
            return bad(KVS_ERR_INVALID, "rows must start on 16-byte boundaries, at least n_head * head_dim apart");
        if (x->x_stride > 1ull << 31 || x->y_stride > 1ull << 31) return bad(KVS_ERR_INVALID, "row stride too large");
        if (norm && !aligned(x->weight, 16)) return bad(KVS_ERR_INVALID, "weight must be 16-byte aligned");
        p.side[i] = {x->x, x->y, (int64_t)x->x_stride, (int64_t)x->y_stride, (int)x->n_head, (int)((x->n_head + heads_a_step - 1) / heads_a_step), norm ? x->weight : nullptr};
    }
    if (n && (!positions || !aligned(positions, position_bytes))) return bad(KVS_ERR_INVALID, "positions null or misaligned");
    if (n > 0x7fffffffull) return bad(KVS_ERR_INVALID, "too many rows");
    if (n == 0) return KVS_OK;
    const int steps = p.side[0].steps + p.side[1].steps;
    const uint64_t fill = (uint64_t)current_device_sms() * 32;  // jobs that fill the card's warp slots
    p.per = (int)((n * steps + fill - 1) / fill);
    if (p.per > steps) p.per = steps;
    p.jobs = (steps + p.per - 1) / p.per;
    p.turns = r->turns;
    p.pos = positions;
    p.wide_pos = position_bytes == 8;
    p.n = (int64_t)n;
    p.rot = (int)r->rot_dim;
    p.interleaved = r->interleaved != 0;
    p.magnitude = r->magnitude;
    p.weight_type = weight_dtype;
    p.eps = eps;
    const uint64_t blocks = (n * p.jobs + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > 0x7fffffffull) return bad(KVS_ERR_UNSUPPORTED, "too many rows for one launch");
    auto kernel = norm ? (D == 64 ? kernel_for<64, true>(dtype) : D == 128 ? kernel_for<128, true>(dtype) : kernel_for<256, true>(dtype))
                       : (D == 64 ? kernel_for<64, false>(dtype) : D == 128 ? kernel_for<128, false>(dtype) : kernel_for<256, false>(dtype));
    void *args[] = {&p};
    const cudaError_t e = cudaLaunchKernel(reinterpret_cast<const void *>(kernel), dim3((unsigned)blocks), dim3(kThreads), args, 0, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) {
        cudaGetLastError();  // the call's own: no later one is to find it
        return bad(KVS_ERR_CUDA, (std::string("rotary launch: ") + cudaGetErrorString(e)).c_str());
    }
    return KVS_OK;
}

}  // namespace
}  // namespace kvs

using namespace kvs;

extern "C" kvs_status kvs_rotate(const kvs_rotary *r, const void *positions, uint32_t position_bytes, uint64_t n, int32_t dtype,
                                 const kvs_head_rows *q, const kvs_head_rows *k, void *stream) {
    return rotary_call(r, positions, position_bytes, n, dtype, q, k, false, KVS_F32, 0.f, stream);
}

extern "C" kvs_status kvs_norm_rotate(const kvs_rotary *r, const void *positions, uint32_t position_bytes, uint64_t n, int32_t dtype,
                                      const kvs_head_rows *q, const kvs_head_rows *k, int32_t weight_dtype, float eps, void *stream) {
    return rotary_call(r, positions, position_bytes, n, dtype, q, k, true, weight_dtype, eps, stream);
}
