// Device helpers shared by the operators around a token mixer: the RMS norm with the
// residual's addition (add_rmsnorm.cu), the short convolution (short_conv.cu) and the
// selective scan (ssm_scan.cu, ssm_backward.cu).
#pragma once
#include <type_traits>

#include "ldn_internal.cuh"

namespace ldn {

// N consecutive elements, widened to fp32.  Vectors of 8 / 16 bytes when VEC (the address is
// then a multiple of the vector), single elements otherwise, STEP apart; places at and past
// `valid` read as zero (VEC vectors are wholly inside or wholly outside).
template <int N, bool VEC, int STEP = 1>
__device__ __forceinline__ void load_n(const float *p, float *v, int valid = N * STEP)
{
    if constexpr (VEC) {
        static_assert(N % 4 == 0, "float4 loads");
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 x = valid > 0 ? *reinterpret_cast<const float4 *>(p + i) : make_float4(0.f, 0.f, 0.f, 0.f);
            v[i] = x.x; v[i + 1] = x.y; v[i + 2] = x.z; v[i + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = i * STEP < valid ? p[i * STEP] : 0.f;
    }
}

__device__ __forceinline__ void bf16x2_widen(uint32_t u, float *v)
{
    v[0] = __uint_as_float(u << 16);   // a bf16 is the upper half of its fp32
    v[1] = __uint_as_float(u & 0xffff0000u);
}

template <int N, bool VEC, int STEP = 1>
__device__ __forceinline__ void load_n(const __nv_bfloat16 *p, float *v, int valid = N * STEP)
{
    if constexpr (VEC && N == 8) {
        const uint4 u = valid > 0 ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0, 0, 0, 0);
        bf16x2_widen(u.x, v); bf16x2_widen(u.y, v + 2); bf16x2_widen(u.z, v + 4); bf16x2_widen(u.w, v + 6);
    } else if constexpr (VEC) {
        static_assert(N == 4, "8- or 16-byte loads");
        const uint2 u = valid > 0 ? *reinterpret_cast<const uint2 *>(p) : make_uint2(0, 0);
        bf16x2_widen(u.x, v); bf16x2_widen(u.y, v + 2);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = i * STEP < valid ? __bfloat162float(p[i * STEP]) : 0.f;
    }
}

__device__ __forceinline__ uint32_t bf16x2_pack(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// N consecutive results, each rounded once to the element type; nothing at and past `valid`.
template <int N, bool VEC, int STEP = 1>
__device__ __forceinline__ void store_n(float *p, const float *v, int valid = N * STEP)
{
    if constexpr (VEC) {
        if (valid > 0)
#pragma unroll
            for (int i = 0; i < N; i += 4)
                *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i * STEP < valid) p[i * STEP] = v[i];
    }
}

template <int N, bool VEC, int STEP = 1>
__device__ __forceinline__ void store_n(__nv_bfloat16 *p, const float *v, int valid = N * STEP)
{
    if constexpr (VEC && N == 8) {
        if (valid > 0)
            *reinterpret_cast<uint4 *>(p) = make_uint4(bf16x2_pack(v[0], v[1]), bf16x2_pack(v[2], v[3]),
                                                       bf16x2_pack(v[4], v[5]), bf16x2_pack(v[6], v[7]));
    } else if constexpr (VEC) {
        static_assert(N == 4, "8- or 16-byte stores");
        if (valid > 0)
            *reinterpret_cast<uint2 *>(p) = make_uint2(bf16x2_pack(v[0], v[1]), bf16x2_pack(v[2], v[3]));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i * STEP < valid) p[i * STEP] = __float2bfloat16_rn(v[i]);
    }
}

// 2^x and 1 / x to about one step, results below the normal numbers as zero.
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 ex2(float2 x) { return make_float2(ex2(x.x), ex2(x.y)); }
__device__ __forceinline__ float2 rcp(float2 x) { return make_float2(rcp(x.x), rcp(x.y)); }
__device__ __forceinline__ float2 dup(float x) { return make_float2(x, x); }
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// sigma(x) = 1 / (1 + e^-x): 0 where e^-x overflows.  e^-x = 2^(-x log2 e) with the scaled exponent
// rounded once and log2 e a float, so beside the two instructions' own step e^-x is off by up to
// 1.3 |x| 2^-24 of itself.  That is at most 0.3 2^-24 in sigma and 0.6 2^-24 in x sigma(x), less than
// an output of 1 is rounded by; only results far below 1 (x well under zero) keep fewer digits than
// an exact exponential gives.  Taking both roundings back to first order costs eight instructions a
// pair and 11.3 for 10.2 us at 7 x 777 x 1028 in fp32, and changes no error of the operators by a tenth.
__device__ __forceinline__ float sigmoid_fast(float x) { return rcp(1.f + ex2(-kLog2e * x)); }

// softplus(x) = max(x, 0) + log(1 + e), e = e^-|x| in (0, 1], of two values in packed
// arithmetic.  log(1 + e) = 2 atanh(s) with s = e / (2 + e) <= 1/3; 2 atanh(s) / s is taken as
// the Chebyshev interpolation of degree 4 in s^2 on [0, 1/9], within 8e-9 of it, so a small
// step size keeps its relative accuracy (a logarithm of 1 + e would lose it in rounding 1 + e).
// The exponent's rounding, worth |x| 2^-24 of e, is taken back to first order.
__device__ __forceinline__ float2 softplus_accurate(float2 x)
{
    // past 100 e is zero in fp32
    const float2 ax = make_float2(fminf(fabsf(x.x), 100.f), fminf(fabsf(x.y), 100.f));
    const float2 l2 = dup(-kLog2e);
    const float2 t = __fmul2_rn(ax, l2);
    const float2 lost = __ffma2_rn(ax, l2, make_float2(-t.x, -t.y));
    float2 e = ex2(t);
    e = __ffma2_rn(__fmul2_rn(e, lost), dup(kLn2), e);
    const float2 s = __fmul2_rn(e, rcp(__fadd2_rn(e, dup(2.f))));
    const float2 q = __fmul2_rn(s, s);
    float2 p = dup(0.281577796f);
    p = __ffma2_rn(p, q, dup(0.279651582f));
    p = __ffma2_rn(p, q, dup(0.400245965f));
    p = __ffma2_rn(p, q, dup(0.666663229f));
    p = __ffma2_rn(p, q, dup(2.f));
    float2 m;   // max(x, 0), where a NaN stays one
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(m.x) : "f"(x.x));
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(m.y) : "f"(x.y));
    return __ffma2_rn(s, p, m);
}
__device__ __forceinline__ float softplus_accurate(float x) { return softplus_accurate(make_float2(x, x)).x; }

// N elements as loaded (16 bytes at a time where VEC): what is prefetched is kept so, since
// widening it would wait for it.  Not PACKED: single elements, a word each, for the same reason.
template <typename T, int N, bool PACKED = true>
struct Raw {
    static constexpr int WORDS = !PACKED ? N : N * (int)sizeof(T) / 4 < 1 ? 1 : N * (int)sizeof(T) / 4;
    uint32_t w[WORDS];
    template <bool VEC, int STEP = 1>
    __device__ __forceinline__ void load(const T *p, int valid)
    {
        if constexpr (!PACKED) {
            using Bits = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
#pragma unroll
            for (int i = 0; i < N; ++i)
                w[i] = i * STEP < valid ? *reinterpret_cast<const Bits *>(p + i * STEP) : 0u;
        } else if constexpr (VEC && WORDS >= 4) {
#pragma unroll
            for (int i = 0; i < WORDS; i += 4) {
                const uint4 q = valid > 0 ? reinterpret_cast<const uint4 *>(p)[i / 4] : make_uint4(0, 0, 0, 0);
                w[i] = q.x; w[i + 1] = q.y; w[i + 2] = q.z; w[i + 3] = q.w;
            }
        } else if constexpr (VEC) {
            static_assert(WORDS == 2, "8- or 16-byte loads");
            const uint2 q = valid > 0 ? *reinterpret_cast<const uint2 *>(p) : make_uint2(0, 0);
            w[0] = q.x; w[1] = q.y;
        } else {
            T *e = reinterpret_cast<T *>(w);
#pragma unroll
            for (int i = 0; i < N; ++i) e[i] = i < valid ? p[i] : T(0.f);
        }
    }
    __device__ __forceinline__ void widen(float *v) const
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = __uint_as_float(w[i]);
        } else if constexpr (!PACKED) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = __uint_as_float(w[i] << 16);
        } else if constexpr (N % 2 == 0) {
#pragma unroll
            for (int i = 0; i < N; i += 2) bf16x2_widen(w[i / 2], v + i);
        } else {
            const T *e = reinterpret_cast<const T *>(w);
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = (float)e[i];
        }
    }
};

// x sigma(x) of two values.
__device__ __forceinline__ float2 silu_fast(float2 x)
{
    return __fmul2_rn(x, rcp(__fadd2_rn(ex2(__fmul2_rn(x, dup(-kLog2e))), dup(1.f))));
}

// Sums across the lanes of mask M, M/2, ..., down to LO, of V values a lane, halving the
// values as it goes: a lane whose bit is set in the current mask keeps the upper half.  Where
// lanes outnumber values the rest of the steps add whole values, so several lanes hold the
// same sum.
template <int V, int M, int LO>
__device__ __forceinline__ void reduce_halving(float *v, int lane)
{
    if constexpr (M >= LO) {
        if constexpr (V > 2) {
            const bool up = (lane & M) != 0;
#pragma unroll
            for (int i = 0; i < V / 2; i += 2) {
                const float2 keep = make_float2(up ? v[V / 2 + i] : v[i], up ? v[V / 2 + i + 1] : v[i + 1]);
                const float2 got = make_float2(__shfl_xor_sync(0xffffffffu, up ? v[i] : v[V / 2 + i], M),
                                               __shfl_xor_sync(0xffffffffu, up ? v[i + 1] : v[V / 2 + i + 1], M));
                const float2 t = __fadd2_rn(keep, got);
                v[i] = t.x;
                v[i + 1] = t.y;
            }
            reduce_halving<V / 2, M / 2, LO>(v, lane);
        } else if constexpr (V == 2) {
            const bool up = (lane & M) != 0;
            const float keep = up ? v[1] : v[0], send = up ? v[0] : v[1];
            v[0] = keep + __shfl_xor_sync(0xffffffffu, send, M);
            reduce_halving<1, M / 2, LO>(v, lane);
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], M);
            reduce_halving<1, M / 2, LO>(v, lane);
        }
    }
}

}  // namespace ldn
