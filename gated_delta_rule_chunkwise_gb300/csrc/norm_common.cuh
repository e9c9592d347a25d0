// Pieces shared by the norms over rows (add_rmsnorm.cu, gated_add_rmsnorm*.cu): a block takes a row,
// 8 channels a thread and vector.
#pragma once
#include "mixer_common.cuh"
#include "sm100_ptx.cuh"

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

// Sums over the block of NV <= 4 values, to every thread, for rows that are taken one after another:
// the warps' sums by halving exchanges (six shuffles for three or four values, in place of fifteen or
// twenty), and a warp reads those of the others as vectors instead of exchanging them again.
// sm: cleared by clear_sums, and another one for the row after.
template <int NV> using Sums = float[NV][kMostThreads / 32];
template <int NV> __device__ __forceinline__ void clear_sums(Sums<NV> &sm)
{
    for (int i = threadIdx.x; i < NV * (kMostThreads / 32); i += blockDim.x) (&sm[0][0])[i] = 0.f;
}
template <int NV> __device__ __forceinline__ void row_sums(float *v, Sums<NV> &sm, int nwarps)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if constexpr (NV == 1) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        if (lane == 0) sm[0][warp] = v[0];
    } else {
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = i < NV ? v[i] : 0.f;
        reduce_halving<4, 16, 1>(w, lane);   // lanes 0, 8, 16, 24 hold values 0 to 3
        if ((lane & 7) == 0 && lane < 8 * NV) sm[lane >> 3][warp] = w[0];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float t = 0.f;
#pragma unroll
        for (int q = 0; q < kMostThreads / 32; q += 4)
            if (q < nwarps) {
                const float4 f = *reinterpret_cast<const float4 *>(&sm[i][q]);
                t += (f.x + f.y) + (f.z + f.w);
            }
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

// A thread's 8 channels in packed arithmetic: two a instruction, where the count of instructions is
// what a row costs.
struct V8 {
    float2 p[kE / 2];
    __device__ __forceinline__ float *values() { return &p[0].x; }
    __device__ __forceinline__ const float *values() const { return &p[0].x; }
};
__device__ __forceinline__ V8 operator*(const V8 &a, const V8 &b)
{
    V8 r;
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) r.p[i] = __fmul2_rn(a.p[i], b.p[i]);
    return r;
}
__device__ __forceinline__ V8 operator*(const V8 &a, float b)
{
    V8 r;
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) r.p[i] = __fmul2_rn(a.p[i], dup(b));
    return r;
}
__device__ __forceinline__ V8 fma(const V8 &a, const V8 &b, const V8 &c)
{
    V8 r;
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) r.p[i] = __ffma2_rn(a.p[i], b.p[i], c.p[i]);
    return r;
}
__device__ __forceinline__ V8 fma(const V8 &a, float b, const V8 &c)
{
    V8 r;
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) r.p[i] = __ffma2_rn(a.p[i], dup(b), c.p[i]);
    return r;
}
// sum + the products' sum, in two chains
__device__ __forceinline__ float2 dot(const V8 &a, const V8 &b, float2 sum)
{
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) sum = __ffma2_rn(a.p[i], b.p[i], sum);
    return sum;
}
__device__ __forceinline__ V8 filled(float x)
{
    V8 r;
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) r.p[i] = dup(x);
    return r;
}
__device__ __forceinline__ V8 sigmoid(const V8 &a)
{
    V8 r;
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) r.p[i] = rcp(__fadd2_rn(ex2(__fmul2_rn(a.p[i], dup(-kLog2e))), dup(1.f)));
    return r;
}
__device__ __forceinline__ V8 as_stored(V8 a, const float *) { return a; }
__device__ __forceinline__ V8 as_stored(V8 a, const __nv_bfloat16 *)
{
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) bf16x2_widen(bf16x2_pack(a.p[i].x, a.p[i].y), &a.p[i].x);
    return a;
}
// A thread's 8 channels in and out of memory, of which those before `valid` are there.  Single elements
// of a thread that has all of them take no comparisons (a warp of a row's inside).
template <bool VEC> __device__ __forceinline__ V8 load8(const float *p, int valid)
{
    V8 r;
    load_n<kE, VEC, kStep<VEC>>(p, r.values(), valid);
    return r;
}
template <bool VEC, typename T> __device__ __forceinline__ void store8(T *p, const V8 &v, int valid)
{
    if (!VEC && valid >= kE * kStep<VEC>) store_n<kE, VEC, kStep<VEC>>(p, v.values());
    else store_n<kE, VEC, kStep<VEC>>(p, v.values(), valid);
}
template <bool VEC, typename R, typename T> __device__ __forceinline__ void take8(R &raw, const T *p, int valid)
{
    if (!VEC && valid >= kE * kStep<VEC>) raw.template load<VEC, kStep<VEC>>(p, kE * kStep<VEC>);
    else raw.template load<VEC, kStep<VEC>>(p, valid);
}
template <typename R> __device__ __forceinline__ V8 widened(const R &raw)
{
    V8 r;
    raw.widen(r.values());
    return r;
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

// ---- rows through a ring in shared memory ----
// A row of registers a thread holds too few bytes on their way for the memory's latency; a ring of rows
// in shared memory, filled by bulk copies, holds as many as fit.  Each stage is one row of each of several
// arrays; the first warps share the copies' issue, which is between two rows' work.
constexpr int kRingMost = 8;                  // stages
constexpr int kRingBytes = 222 * 1024;        // of an SM, beside the kernels' static arrays
constexpr uint64_t kRingWaitNs = 2000000000ull;

struct RingPlan {
    int stages, stage;   // rows, bytes of one
};

// Stages for `blocks` blocks an SM of rows of `bytes`; 0 where a ring would not hold two rows.
inline RingPlan ring_plan(int bytes, int blocks)
{
    const int n = std::min(kRingMost, kRingBytes / blocks / bytes);
    return {n < 2 ? 0 : n, bytes};
}

// ARRAYS: how many; one of rows of no bytes is left out.
template <int ARRAYS> struct RowRing {
    uint8_t *base;
    uint64_t *full;
    int *fail;
    int stages, stage, issuers, s = 0;
    uint32_t phase = 0, own = 0, mine = 0;   // arrays that this warp issues, a bit each, and their bytes of a row
    const char *from[ARRAYS];
    int bytes[ARRAYS];

    // Every thread; `bars`: kRingMost barriers in shared memory.  __syncthreads() before the first use.
    __device__ __forceinline__ RowRing(uint8_t *smem, uint64_t *bars, int *failed, RingPlan p)
        : base(smem), full(bars), fail(failed), stages(p.stages), stage(p.stage),
          issuers(min(ARRAYS, (int)blockDim.x >> 5))
    {
        if (threadIdx.x == 0) {
            *fail = 0;
            for (int i = 0; i < stages; ++i) sm100::mbar_init(full + i, issuers);
            sm100::fence_mbar_init();
        }
    }
    // Array I has rows of `size` bytes (a multiple of 16, as its address is), after I - 1's; its place in
    // a stage.
    template <int I> __device__ __forceinline__ int add(const void *p, int size)
    {
        int at = 0;
#pragma unroll
        for (int i = 0; i < I; ++i) at += bytes[i];
        from[I] = (const char *)p;
        bytes[I] = size;
        if (size && I % issuers == (int)(threadIdx.x >> 5)) {
            own |= 1u << I;
            mine += size;
        }
        return at;
    }
    // Whether this thread issues copies: then it calls fill, as the other issuers do.
    __device__ __forceinline__ bool issues() const { return (threadIdx.x & 31) == 0 && (int)threadIdx.x < 32 * issuers; }
    // Row `row` of every array into stage `to`.
    __device__ __forceinline__ void fill(int to, long long row)
    {
        sm100::mbar_arrive_expect_tx(full + to, mine);
        uint8_t *d = base + (size_t)to * stage;
#pragma unroll
        for (int i = 0; i < ARRAYS; ++i) {
            if (own >> i & 1) sm100::bulk_load(d, from[i] + row * bytes[i], bytes[i], full + to);
            d += bytes[i];
        }
    }
    // The current stage, once it has arrived; after a wait that ran out, at once.
    __device__ __forceinline__ const uint8_t *row()
    {
        if (!*(volatile int *)fail && !sm100::mbar_wait(full + s, phase, kRingWaitNs)) *(volatile int *)fail = 1;
        return base + (size_t)s * stage;
    }
    __device__ __forceinline__ void step()
    {
        if (++s == stages) {
            s = 0;
            phase ^= 1;
        }
    }
    // Every thread, at the end: nothing is left under way, and a wait that ran out is recorded.
    __device__ __forceinline__ void close(int *status)
    {
        __syncthreads();
        if (threadIdx.x == 0 && *fail) {
            atomicOr(status, 1 << LDN_ERR_TIMEOUT);
            for (int i = 0; i < stages; ++i)   // whichever phase a stage is in, the other one is over
                sm100::mbar_wait(full + i, phase ^ (i < s), kRingWaitNs / 8);
        }
        __syncthreads();
    }
};

}  // namespace
}  // namespace ldn
