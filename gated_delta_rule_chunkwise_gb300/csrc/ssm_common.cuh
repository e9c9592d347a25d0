// Pieces of the selective scan shared by its directions: a tile's rows on their way to shared
// memory, and the decay rates.
#pragma once
#include "mixer_common.cuh"
#include "sm100_ptx.cuh"

namespace ldn {
namespace ssm {
using sm100::cp_async_commit;
using sm100::cp_async_wait;

constexpr int TT = kSsmChunk;   // tokens of a tile

// Copies BYTES (4, 8 or 16) from global to shared memory, or zeros where `ok` is false; in flight
// until its group is waited for.
template <int BYTES>
__device__ __forceinline__ void cp_async(void *dst, const void *src, bool ok)
{
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst), n = ok ? BYTES : 0;
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(d), "l"(src), "r"(n), "n"(BYTES)
                     : "memory");
}

// The tile's rows of one warp's WC channels, to dst[TT][WC], by that warp; zeros outside.
// FULL: nothing is outside.
template <typename T, int WC, bool VEC, bool FULL>
__device__ __forceinline__ void warp_rows(T *dst, const T *src, long long ld, int rows, int cols)
{
    constexpr int E = VEC ? (WC * (int)sizeof(T) < 16 ? WC : 16 / (int)sizeof(T)) : 1, PER = WC / E;
#pragma unroll
    for (int k = 0; k < TT * PER / 32; ++k) {
        const int i = k * 32 + (int)(threadIdx.x & 31), r = i / PER, e = (i % PER) * E;
        const bool ok = FULL || (r < rows && e < cols);
        if constexpr (VEC) cp_async<E * (int)sizeof(T)>(dst + i * E, ok ? src + r * ld + e : src, ok);
        else dst[i] = ok ? src[r * ld + e] : T(0.f);
    }
}

// A tile's B or C rows by NT threads: copied one tile ahead, then widened by the threads that
// copied them to dst[TT][N], with zeros at and past `rows`.  A thread takes K neighbouring
// elements, in whole vectors or 4-byte words as the rows are aligned; a projection's slices
// may start at any element, and rows that are not aligned to words are read where they are
// widened.
template <typename T, int N, int NT>
struct SharedRows {
    static constexpr int MOST = 16 / (int)sizeof(T), PER = TT * N / NT;
    static constexpr int K = PER < 4 ? 4 : PER < MOST ? PER : MOST;
    static constexpr int TURNS = (TT * N + NT * K - 1) / (NT * K), BYTES = K * (int)sizeof(T);
    enum { kSingles, kWords, kVectors };
    static __device__ __forceinline__ void fetch(T *raw, const T *src, long long ld, int rows, int how, int tid)
    {
        if (how == kSingles) return;
#pragma unroll
        for (int k = 0; k < TURNS; ++k) {
            const int i = (k * NT + tid) * K, r = i / N;
            if (TT * N % (NT * K) != 0 && i >= TT * N) continue;
            const bool ok = r < rows;
            const T *p = ok ? src + r * ld + i % N : src;
            if (how == kVectors) cp_async<BYTES>(raw + i, p, ok);
            else
#pragma unroll
                for (int c = 0; c < K; c += 4 / (int)sizeof(T)) cp_async<4>(raw + i + c, ok ? p + c : p, ok);
        }
    }
    static __device__ __forceinline__ void widen(float *dst, const T *raw, const T *src, long long ld, int rows,
                                                 int how, int tid)
    {
#pragma unroll
        for (int k = 0; k < TURNS; ++k) {
            const int i = (k * NT + tid) * K, r = i / N;
            if (TT * N % (NT * K) != 0 && i >= TT * N) continue;
            float v[K];
            if (how == kSingles) load_n<K, false>(src + r * ld + i % N, v, r < rows ? K : 0);
            else load_n<K, true>(raw + i, v);
#pragma unroll
            for (int c = 0; c < K; c += 4)
                *reinterpret_cast<float4 *>(dst + i + c) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
        }
    }
    static __device__ __forceinline__ int alignment(const T *p, long long ld)
    {
        const uintptr_t m = (uintptr_t)p | (uintptr_t)(ld * (long long)sizeof(T));
        return m % BYTES == 0 ? kVectors : m % 4 == 0 ? kWords : kSingles;
    }
};

// A log2 e, finite: -infinity forgets whatever the step, but a row behind a sequence's end steps
// by zero and keeps the state.
__device__ __forceinline__ float rate(float A)
{
    float r;
    asm("max.NaN.f32 %0, %1, 0fff7fffff;" : "=f"(r) : "f"(A * kLog2e));
    return r;
}

// e^{dt A} = 2^{dt A2} of rates A2 = rate(A).  The approximation of 2^x is low by 0.35 x 2^-24 on
// average for x in (-1, 0) (measured), and a decay near 1 compounds that over its memory: an
// exponent of 2^-25 more takes the mean off for nothing, the product being a fused one.  2^0
// stays 1: the instruction has no value between 1 and 1 + 2^-23.
constexpr float kMean = 0x1p-25f;
__device__ __forceinline__ float2 decay(float2 A2, float dt) { return ex2(__ffma2_rn(A2, dup(dt), dup(kMean))); }
__device__ __forceinline__ float decay(float A2, float dt) { return ex2(fmaf(A2, dt, kMean)); }

__device__ __forceinline__ int seq_len(const int *lens, int b, int T)
{
    return lens ? min(max(lens[b], 0), T) : T;
}

}  // namespace ssm
}  // namespace ldn
