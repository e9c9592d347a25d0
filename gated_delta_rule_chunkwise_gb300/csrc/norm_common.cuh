// Pieces shared by the norms over rows (add_rmsnorm.cu, gated_add_rmsnorm*.cu): a block takes a row,
// 8 channels a thread and vector.
#pragma once
#include "mixer_common.cuh"

namespace ldn {
namespace {

constexpr int kE = 8;   // channels per thread and vector
constexpr int kMostThreads = 512;

// Sums over the block, to every thread, through sm[32 NV].
template <int NV>
__device__ __forceinline__ void block_sum(float *v, float *sm, int nwarps)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < NV; ++i) sm[i * 32 + warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float t = lane < nwarps ? sm[i * 32 + lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        v[i] = t;
    }
}

// A thread's place in a vector of the block's, and the distance of its 8 channels: consecutive
// where rows are whole 16-byte vectors; otherwise 32 apart, so that a warp takes the same 256
// channels and its single elements are neighbours (5000 x 777 in bf16: 9.8 us for 22.5 with
// consecutive ones, gradient 13.4 for 18.2).
template <bool VEC> constexpr int kStep = VEC ? 1 : 32;
template <bool VEC> __device__ __forceinline__ int place(int k, int t)
{
    return k * (int)blockDim.x * kE + (VEC ? t * kE : (t & ~31) * kE + (t & 31));
}

template <bool VEC> __device__ __forceinline__ int place(int k) { return place<VEC>(k, (int)threadIdx.x); }

// Rounds to the stored type and back.
__device__ __forceinline__ float as_stored(float x, const float *) { return x; }
__device__ __forceinline__ float as_stored(float x, const __nv_bfloat16 *)
{
    return __bfloat162float(__float2bfloat16_rn(x));
}

// 1 / sqrt(v) to about half a step: rsqrtf's two and a half, taken back to first order.
__device__ __forceinline__ float root(float v)
{
    const float r = rsqrtf(v), e = fmaf(-v * r, r, 1.f);
    return fabsf(e) < 1.f ? fmaf(0.5f * r, e, r) : r;   // r where v is 0, infinite or NaN
}

// Threads for D channels at vpt vectors of 8 each, in whole warps.
inline int norm_threads(int D, int vpt) { return std::min(kMostThreads, (((D + kE * vpt - 1) / (kE * vpt) + 31) / 32) * 32); }

inline bool vec16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace
}  // namespace ldn
