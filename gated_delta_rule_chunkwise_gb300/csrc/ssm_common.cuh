// Pieces of the selective scan shared by its directions: the tile of a token run in shared
// memory and the packed arithmetic.
#pragma once
#include "mixer_common.cuh"
#include "sm100_ptx.cuh"

namespace ldn {
namespace ssm {
using sm100::cp_async16;
using sm100::cp_async_commit;
using sm100::cp_async_wait;

constexpr int TT = kSsmChunk;   // tokens of a tile
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 ex2(float2 x) { return make_float2(ex2(x.x), ex2(x.y)); }
__device__ __forceinline__ float2 dup(float x) { return make_float2(x, x); }

// Rows t0 .. t0 + TT of DB channels to dst[TT][DB]; rows at and past `rows` and channels at
// and past `cols` are zeros.  VEC: 16-byte copies, in flight until their group is waited for.
template <typename T, int DB, int NT, bool VEC>
__device__ __forceinline__ void load_rows(T *dst, const T *src, long long ld, int rows, int cols)
{
    if constexpr (VEC) {
        constexpr int E = 16 / sizeof(T), PER = DB / E;
        for (int i = threadIdx.x; i < TT * PER; i += NT) {
            const int r = i / PER, e = (i % PER) * E;
            const bool ok = r < rows && e < cols;
            cp_async16(dst + r * DB + e, ok ? src + r * ld + e : src, ok ? 16u : 0u);
        }
    } else {
        for (int i = threadIdx.x; i < TT * DB; i += NT) {
            const int r = i / DB, e = i % DB;
            dst[i] = r < rows && e < cols ? src[r * ld + e] : T(0.f);
        }
    }
}

// A run's B or C rows, widened, to dst[TT][N]; zeros at and past `rows`.  The rows are single
// elements to the loads: a projection's slices start at any element.
template <typename T, int N, int NT>
struct RowRegs {
    static constexpr int K = (TT * N + NT - 1) / NT;
    T v[K];
    __device__ __forceinline__ void load(const T *src, long long ld, int rows)
    {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = k * NT + (int)threadIdx.x, r = i / N;
            v[k] = r < rows && (TT * N % NT == 0 || i < TT * N) ? src[r * ld + i % N] : T(0.f);
        }
    }
    __device__ __forceinline__ void store(float *dst) const
    {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = k * NT + (int)threadIdx.x;
            if (TT * N % NT == 0 || i < TT * N) dst[i] = (float)v[k];
        }
    }
};

__device__ __forceinline__ int seq_len(const int *lens, int b, int T)
{
    return lens ? min(max(lens[b], 0), T) : T;
}

}  // namespace ssm
}  // namespace ldn
