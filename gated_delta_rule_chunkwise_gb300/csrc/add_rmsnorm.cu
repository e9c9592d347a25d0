// RMS norm with the residual's addition, and its gradient.
//
//   s = x + r (stored in the residual's type),  rstd = 1 / sqrt(mean_c s_c^2 + eps),
//   y = s rstd w,   as the element type or in e4m3 with scales:
//   scale = max(max_group |y|, 2^-100) / 448,  q = e4m3(y / scale), saturating;
//   a group is 128 consecutive channels or the whole row.  y and scale are fp32; q is rounded as the
//   quotient in 64 bits, stored in fp32, would be.
// The norm is taken of s AS STORED: a bf16 residual stream rounds the sum once, and that
// value is what the next block adds to and what the gradient reads back.
//
//   ds = dsum + rstd (w dy - s rstd^2 mean_c(w dy s)),  dw = sum over rows of dy s rstd.
//
// Both directions move every byte once and are bound by HBM: a row lives in registers (8
// channels a thread and vector), two block sums a row.  Arithmetic is fp32.  16384 x 4096 in
// bf16 to e4m3 takes 72.5 us by rows and 75.6 by 128 (6,480 and 6,240 GB/s), 8192 x 2048 with an fp32
// residual stream 31.5 and the gradient 43.8 (6,380 and 6,130 GB/s).  Rows past 8192 channels have
// more vectors a thread than registers for a next row, and at eight some spill: 4096 x 16384 94 us
// (5,690 GB/s; e4m3 83 and 107), 2048 x 32768 92, and the gradient, with nothing on its way, 265
// (2,030 GB/s).
#include <cuda_fp8.h>

#include "norm_common.cuh"

namespace ldn {
namespace {

// An SM's threads in the row walk: 1024 to e4m3 by rows, where a row near a border holds its block
// up (16384 x 4096: 89 us at 512, 75.6 at 768, 72.5 at 1024, 93 at 1280; 8192 x 8192 73 for 93 at
// 768), 768 otherwise (16384 x 4096 by 128: 75.6 us, 92 at 1024 with the registers it has; as the
// element type 84, 88 at 1024).
constexpr int norm_threads_sm(int eight) { return eight == 1 ? 1024 : 768; }
constexpr float kE4m3Max = 448.f, kLeast = 0x1p-100f;   // kLeast: of a group's largest |y|

// The largest value over the block, to every thread, through sm[32]; `at` gets every warp's lane that
// holds its largest.
__device__ __forceinline__ float block_max(float v, float *sm, int *at, int nwarps)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float t = v;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
    const unsigned holds = __ballot_sync(0xffffffffu, v == t);
    if (lane == 0) {
        sm[warp] = t;
        at[warp] = __ffs(holds) - 1;
    }
    __syncthreads();
    t = lane < nwarps ? sm[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
    return t;
}

template <int N, bool VEC, int STEP>
__device__ __forceinline__ void store_e4m3(uint8_t *p, const float *v, int valid)
{
    static_assert(N == 8, "two words");
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]), __NV_SATFINITE,
                                                     __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    if constexpr (VEC) {
        if (valid > 0) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i * STEP < valid) p[i * STEP] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
    }
}

// ---- e4m3 ----
// y / scale = 448 |s w| / max |s w|: rstd drops out, but where the group's largest |y| is below the
// least.  m is the largest |s w|.
__device__ __forceinline__ float scale_up(float m, float rstd)
{
    return m * rstd > kLeast ? kE4m3Max / m : kE4m3Max / kLeast * rstd;   // NaN where rstd is
}

// In fp32 that quotient is off by up to four roundings (both products', the division's, the last
// product's).  They matter only where it lies so near the middle of two neighbours in e4m3: the 20 bits
// that are rounded away are then within kNear steps of their half (one value in 95,000, and every value
// that is halfway exactly: rows of equal weights have such).  There it is decided as a quotient in 64
// bits, stored in fp32, would be: 448 |s w| against the middle times max |s w|, both as exact sums of two
// floats.  Values below e4m3's normal numbers stay with fp32.
constexpr uint32_t kNear = 5;
__device__ __forceinline__ uint32_t from_border(float v)   // up to 2 kNear << 12 where near
{
    return (__float_as_uint(v) << 12) + (0x80000000u + (kNear << 12));
}
__device__ __forceinline__ bool near_border(uint32_t t) { return t <= kNear << 13; }

struct Pair { float hi, lo; };   // a sum of two floats, hi the nearest to it
__device__ __forceinline__ Pair product(float a, float b)
{
    const float p = __fmul_rn(fabsf(a), fabsf(b));
    return {p, __fmaf_rn(fabsf(a), fabsf(b), -p)};
}
__device__ __forceinline__ Pair larger(Pair a, Pair b)
{
    return b.hi > a.hi || (b.hi == a.hi && b.lo > a.lo) ? b : a;
}
__device__ __forceinline__ Pair largest(Pair a, int lanes)   // over groups of lanes
{
    for (int o = lanes / 2; o > 0; o >>= 1)
        a = larger(a, {__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)});
    return a;
}
// v moved to its side of the border that it is near: the middle, or a step of fp32 beside it, where
// p is |s w| and `top` the largest.
__device__ __forceinline__ float settled(float v, Pair p, Pair top)
{
    const uint32_t bits = __float_as_uint(v), middle = (bits & 0xfff00000u) | 0x80000u;
    const float b = fabsf(__uint_as_float(middle)), c = b * top.hi;
    const float half = __uint_as_float(bits & 0x7f800000u) * 0x1p-24f * top.hi;   // half a step of fp32
    // the first two differences are exact: what they are of is equal to 20 bits
    const float d = (fmaf(kE4m3Max, p.hi, -c) - fmaf(b, top.hi, -c)) + fmaf(kE4m3Max, p.lo, -b * top.lo);
    if (!(p.hi > 0x1p-90f && top.hi < 0x1p90f)) return v;   // no ordinary numbers
    return __uint_as_float(middle + (d > half) - (d < -half));
}

// The thread's values of a row near a border, once all are stored (a warp together; s: the row as
// stored).  Everything is formed again from memory: registers kept for one row in twenty would cost
// every row a third of its warps.  EIGHT = 1: the row's largest |s w| is `top`, of thread `owner`.
template <typename T, int EIGHT, bool VEC, int STEP>
__device__ __forceinline__ void settle_row(const T *s, const float *w, uint8_t *q, int vectors, int D, float rstd,
                                           float top, int owner)
{
    constexpr int N = EIGHT == 2 && !VEC ? 4 : kE, LANES = VEC ? 16 : 32;   // a lane's channels of a group, its lanes
    auto value = [](float a, float g, float up) { return __fmul_rn(__fmul_rn(a, g), up); };   // as in the walk
    Pair most{0.f, 0.f};
    bool found = false;
#pragma unroll 1
    for (int k = 0; k < vectors * (kE / N); ++k) {
        const int c = place<VEC>(k / (kE / N)) + k % (kE / N) * N * STEP;
        float a[N], g[N];
        load_n<N, VEC, STEP>(s + c, a, D - c);
        load_n<N, VEC, STEP>(w + c, g, D - c);
        if constexpr (EIGHT == 2) {
            top = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) top = fmaxf(top, fabsf(__fmul_rn(a[i], g[i])));
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        }
        const float up = scale_up(top, rstd);
        unsigned near = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) near |= (unsigned)near_border(from_border(value(a[i], g[i], up))) << i;
        if (!__any_sync(0xffffffffu, near != 0)) continue;
        if constexpr (EIGHT == 2) {
            most = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < N; ++i) most = larger(most, product(a[i], g[i]));
            most = largest(most, LANES);
        } else if (!found) {
            // the largest is the owner's, unless another rounds to the same
#pragma unroll 1
            for (int i = threadIdx.x & 31; i < vectors * kE; i += 32) {
                const int at = place<VEC>(i / kE, owner) + i % kE * STEP;
                if (at < D) {
                    const Pair p = product((float)s[at], w[at]);
                    if (p.hi == top) most = larger(most, p);
                }
            }
            most = largest(most, 32);
            found = true;
        }
        if (!(top * rstd > kLeast)) continue;
#pragma unroll 1
        for (; near; near &= near - 1) {
            const int at = c + (__ffs(near) - 1) * STEP;
            const float x = (float)s[at], f = w[at], v = value(x, f, up);
            if (fabsf(v) < 2.f * kE4m3Max)
                q[at] = (uint8_t)__nv_cvt_float_to_fp8(settled(v, product(x, f), most), __NV_SATFINITE, __NV_E4M3);
        }
    }
}

// In the walk's own code where a row's neighbours are in registers meanwhile; where none are, a call
// leaves more of them to the walk (2000 x 20001 by rows: 188 us inlined, 155 called).
template <typename T, int EIGHT, bool VEC, int STEP>
__device__ __noinline__ void settle_called(const T *s, const float *w, uint8_t *q, int vectors, int D, float rstd,
                                           float top, int owner)
{
    settle_row<T, EIGHT, VEC, STEP>(s, w, q, vectors, D, rstd, top, owner);
}
template <typename T, int EIGHT, bool VEC, int STEP, bool INLINE>
__device__ __forceinline__ void settle(const T *s, const float *w, uint8_t *q, int vectors, int D, float rstd, float top,
                                       int owner)
{
    if constexpr (INLINE) settle_row<T, EIGHT, VEC, STEP>(s, w, q, vectors, D, rstd, top, owner);
    else settle_called<T, EIGHT, VEC, STEP>(s, w, q, vectors, D, rstd, top, owner);
}

// EIGHT: 0 = y in TIn, 1 = e4m3 with a scale per row, 2 = per 128 channels.  A block walks rows
// blockIdx.x, + gridDim.x, ...; the next row is on its way while one is summed and stored.
template <typename TIn, typename TRes, int EIGHT, int VPT, bool VEC>
__global__ void __launch_bounds__(kMostThreads)
add_rmsnorm_kernel(const TIn *__restrict__ x, const TRes *r, const float *__restrict__ w, void *__restrict__ y,
                   float *__restrict__ scale, TRes *r_out, long long rows, int D, float eps)
{
    __shared__ float sm[2][64];
    __shared__ int at[EIGHT == 1 ? 2 : 1][EIGHT == 1 ? 16 : 1];
    const int nt = blockDim.x, nwarps = nt >> 5;
    constexpr bool KEEP = VPT <= 2;   // the weights stay in registers, the next row comes ahead
    float g[KEEP ? VPT : 1][kE];
    if constexpr (KEEP)
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = place<VEC>(k);
            load_n<kE, VEC, kStep<VEC>>(w + c, g[k], D - c);
        }
    Raw<TIn, kE, VEC> rx[VPT];
    Raw<TRes, kE, VEC> rr[VPT];
    auto fetch = [&](long long row) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = place<VEC>(k), valid = row < rows ? D - c : 0;
            rx[k].template load<VEC, kStep<VEC>>(x + row * D + c, valid);
            rr[k].template load<VEC, kStep<VEC>>(r + (r ? row * D + c : 0), r ? valid : 0);
        }
    };
    fetch(blockIdx.x);
    int turn = 0;
    for (long long row = blockIdx.x; row < rows; row += gridDim.x, turn ^= 1) {
        float v[VPT][kE], ss = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = place<VEC>(k);
            rx[k].widen(v[k]);
            if (r) {
                float q[kE];
                rr[k].widen(q);
#pragma unroll
                for (int i = 0; i < kE; ++i) v[k][i] = as_stored(v[k][i] + q[i], r);
                store_n<kE, VEC, kStep<VEC>>(r_out + row * D + c, v[k], D - c);
            }
#pragma unroll
            for (int i = 0; i < kE; ++i) ss = fmaf(v[k][i], v[k][i], ss);
        }
        if constexpr (KEEP) fetch(row + gridDim.x);
        block_sum<1>(&ss, sm[turn], nwarps);   // two buffers: the next row's sums pass no reader of these
        const float rstd = rsqrtf(ss / (float)D + eps);
        float top = 0.f;
        uint32_t near = 0xffffffffu;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = place<VEC>(k), valid = D - c;
            if constexpr (!KEEP) load_n<kE, VEC, kStep<VEC>>(w + c, g[0], valid);
#pragma unroll
            for (int i = 0; i < kE; ++i)
                v[k][i] = EIGHT ? __fmul_rn(v[k][i], g[KEEP ? k : 0][i]) : v[k][i] * (rstd * g[KEEP ? k : 0][i]);
            if constexpr (EIGHT == 0) {
                store_n<kE, VEC, kStep<VEC>>((TIn *)y + row * D + c, v[k], valid);
            } else {
                float m = 0.f;
                if constexpr (EIGHT == 1 || VEC)
#pragma unroll
                    for (int i = 0; i < kE; ++i) m = fmaxf(m, fabsf(v[k][i]));
                if constexpr (EIGHT == 2 && !VEC) {
                    // 128 channels are four of every lane's
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        m = 0.f;
#pragma unroll
                        for (int i = 4 * h; i < 4 * h + 4; ++i) m = fmaxf(m, fabsf(v[k][i]));
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                        const float up = scale_up(m, rstd);
#pragma unroll
                        for (int i = 4 * h; i < 4 * h + 4; ++i) near = min(near, from_border(v[k][i] = __fmul_rn(v[k][i], up)));
                        if ((threadIdx.x & 31) == 0 && valid > 128 * h)
                            scale[row * (long long)((D + 127) / 128) + c / 128 + h] = fmaxf(m * rstd, kLeast) / kE4m3Max;
                    }
                    store_e4m3<kE, VEC, kStep<VEC>>((uint8_t *)y + row * D + c, v[k], valid);
                } else if constexpr (EIGHT == 2) {
                    // 128 channels are the 8-channel vectors of 16 neighbouring lanes
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                    const float up = scale_up(m, rstd);
#pragma unroll
                    for (int i = 0; i < kE; ++i) near = min(near, from_border(v[k][i] = __fmul_rn(v[k][i], up)));
                    store_e4m3<kE, VEC, kStep<VEC>>((uint8_t *)y + row * D + c, v[k], valid);
                    if ((threadIdx.x & 15) == 0 && valid > 0)
                        scale[row * (long long)((D + 127) / 128) + c / 128] = fmaxf(m * rstd, kLeast) / kE4m3Max;
                } else {
                    top = fmaxf(top, m);
                }
            }
        }
        if constexpr (EIGHT == 1) {
            top = block_max(top, sm[turn] + 32, at[turn], nwarps);
            const float up = scale_up(top, rstd);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = place<VEC>(k);
#pragma unroll
                for (int i = 0; i < kE; ++i) near = min(near, from_border(v[k][i] = __fmul_rn(v[k][i], up)));
                store_e4m3<kE, VEC, kStep<VEC>>((uint8_t *)y + row * D + c, v[k], D - c);
            }
            if (threadIdx.x == 0) scale[row] = fmaxf(top * rstd, kLeast) / kE4m3Max;
        }
        if constexpr (EIGHT != 0)
            if (__any_sync(0xffffffffu, near_border(near))) {
                uint8_t *q = (uint8_t *)y + row * D;
                int owner = 0;
                if constexpr (EIGHT == 1) {
                    const int lane = threadIdx.x & 31;
                    const unsigned holds = __ballot_sync(0xffffffffu, lane < nwarps && sm[turn][32 + lane] == top);
                    owner = holds ? (__ffs(holds) - 1) * 32 + at[turn][__ffs(holds) - 1] : 0;
                }
                if (std::is_same_v<TIn, TRes> || r)
                    settle<TRes, EIGHT, VEC, kStep<VEC>, KEEP>(r ? r_out + row * D : (const TRes *)x + row * D, w, q, VPT, D,
                                                               rstd, top, owner);
                else
                    settle<TIn, EIGHT, VEC, kStep<VEC>, KEEP>(x + row * D, w, q, VPT, D, rstd, top, owner);
            }
        if constexpr (!KEEP) fetch(row + gridDim.x);
    }
}

// A block walks rows blockIdx.x, + gridDim.x, ...; the next row is on its way while one is
// summed.  The columns' share of dw stays in registers over all rows and goes to `part`
// [gridDim.x][D] once.
template <typename TIn, typename TRes, int VPT, bool VEC>
__global__ void __launch_bounds__(kMostThreads)
add_rmsnorm_bwd_kernel(const TIn *__restrict__ dy, const TRes *__restrict__ s, const float *__restrict__ w,
                       const TRes *__restrict__ dsum, TIn *__restrict__ dx, TRes *__restrict__ dres,
                       float *__restrict__ part, long long rows, int D, float eps)
{
    __shared__ float sm[2][64];
    const int nt = blockDim.x, nwarps = nt >> 5;
    float acc[VPT][kE], g[VPT][kE];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int c = place<VEC>(k);
        load_n<kE, VEC, kStep<VEC>>(w + c, g[k], D - c);
#pragma unroll
        for (int i = 0; i < kE; ++i) acc[k][i] = 0.f;
    }
    constexpr int AHEAD = VPT == 1 ? 2 : 1;   // rows on their way: as many as there are registers for
    Raw<TRes, kE, VEC> rs[AHEAD][VPT], rd[AHEAD][VPT];
    Raw<TIn, kE, VEC> ry[AHEAD][VPT];
    auto fetch = [&](int h, long long row) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = place<VEC>(k), valid = row < rows ? D - c : 0;
            rs[h][k].template load<VEC, kStep<VEC>>(s + row * D + c, valid);
            ry[h][k].template load<VEC, kStep<VEC>>(dy + row * D + c, valid);
            rd[h][k].template load<VEC, kStep<VEC>>(dsum + row * D + c, dsum ? valid : 0);
        }
    };
    auto one = [&](int h, int turn, long long row) {
        float sv[VPT][kE], gy[VPT][kE], d[VPT][kE], sums[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            rs[h][k].widen(sv[k]);
            ry[h][k].widen(gy[k]);
            rd[h][k].widen(d[k]);
#pragma unroll
            for (int i = 0; i < kE; ++i) {
                sums[0] = fmaf(sv[k][i], sv[k][i], sums[0]);
                sums[1] = fmaf(g[k][i] * gy[k][i], sv[k][i], sums[1]);
            }
        }
        fetch(h, row + (long long)AHEAD * gridDim.x);
        block_sum<2>(sums, sm[turn], nwarps);   // two buffers: the next row's sums pass no reader of these
        const float rstd = rsqrtf(sums[0] / (float)D + eps);
        const float m = rstd * rstd * (sums[1] / (float)D);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = place<VEC>(k), valid = D - c;
#pragma unroll
            for (int i = 0; i < kE; ++i) {
                acc[k][i] = fmaf(gy[k][i], sv[k][i] * rstd, acc[k][i]);
                d[k][i] = fmaf(rstd, g[k][i] * gy[k][i] - sv[k][i] * m, d[k][i]);
            }
            if (dx) store_n<kE, VEC, kStep<VEC>>(dx + row * D + c, d[k], valid);
            if (dres) store_n<kE, VEC, kStep<VEC>>(dres + row * D + c, d[k], valid);
        }
    };
    fetch(0, blockIdx.x);
    if constexpr (AHEAD == 2) fetch(1, blockIdx.x + (long long)gridDim.x);
    for (long long row = blockIdx.x; row < rows; row += 2ll * gridDim.x) {
        one(0, 0, row);
        if (row + gridDim.x < rows) one(AHEAD - 1, 1, row + gridDim.x);
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int c = place<VEC>(k);
        store_n<kE, VEC, kStep<VEC>>(part + (size_t)blockIdx.x * D + c, acc[k], D - c);
    }
}

// out[c] = sum over n rows of part[n][c]: 32 columns a block, kSumRows rows at a time.
constexpr int kSumRows = 32;
__global__ void __launch_bounds__(32 * kSumRows)
column_sum_kernel(const float *__restrict__ part, float *__restrict__ out, int n, int D)
{
    __shared__ float sm[kSumRows][33];
    const int c = blockIdx.x * 32 + threadIdx.x, y = threadIdx.y;
    float t = 0.f;
    if (c < D)
#pragma unroll 8
        for (int i = y; i < n; i += kSumRows) t += part[(size_t)i * D + c];
    sm[y][threadIdx.x] = t;
    __syncthreads();
    if (y == 0 && c < D) {
#pragma unroll
        for (int i = 1; i < kSumRows; ++i) t += sm[i][threadIdx.x];
        out[c] = t;
    }
}

// Rows too wide for registers: s and dy are read again (from L2) after the sums, and the
// columns' share of dw stays in shared memory, each column its thread's own.
template <typename TIn, typename TRes, bool VEC>
__global__ void __launch_bounds__(kMostThreads)
add_rmsnorm_bwd_wide_kernel(const TIn *__restrict__ dy, const TRes *__restrict__ s, const float *__restrict__ w,
                            const TRes *__restrict__ dsum, TIn *__restrict__ dx, TRes *__restrict__ dres,
                            float *__restrict__ part, long long rows, int D, float eps)
{
    extern __shared__ float acc[];
    __shared__ float sm[2][64];
    const int nt = blockDim.x, step = nt * kE, first = place<VEC>(0);
    constexpr int E = kStep<VEC>;   // a thread's channels are c + i E
    for (int c = first; c < D; c += step)
#pragma unroll
        for (int i = 0; i < kE; ++i)
            if (c + i * E < D) acc[c + i * E] = 0.f;
    int turn = 0;
    for (long long row = blockIdx.x; row < rows; row += gridDim.x, turn ^= 1) {
        float sums[2] = {0.f, 0.f}, sv[kE], gy[kE], g[kE], d[kE];
        for (int c = first; c < D; c += step) {
            load_n<kE, VEC, kStep<VEC>>(s + row * D + c, sv, D - c);
            load_n<kE, VEC, kStep<VEC>>(dy + row * D + c, gy, D - c);
            load_n<kE, VEC, kStep<VEC>>(w + c, g, D - c);
#pragma unroll
            for (int i = 0; i < kE; ++i) {
                sums[0] = fmaf(sv[i], sv[i], sums[0]);
                sums[1] = fmaf(g[i] * gy[i], sv[i], sums[1]);
            }
        }
        block_sum<2>(sums, sm[turn], nt >> 5);
        const float rstd = rsqrtf(sums[0] / (float)D + eps);
        const float m = rstd * rstd * (sums[1] / (float)D);
        for (int c = first; c < D; c += step) {
            load_n<kE, VEC, kStep<VEC>>(s + row * D + c, sv, D - c);
            load_n<kE, VEC, kStep<VEC>>(dy + row * D + c, gy, D - c);
            load_n<kE, VEC, kStep<VEC>>(w + c, g, D - c);
            load_n<kE, VEC, kStep<VEC>>(dsum + row * D + c, d, dsum ? D - c : 0);
#pragma unroll
            for (int i = 0; i < kE; ++i) {
                if (c + i * E < D) acc[c + i * E] = fmaf(gy[i], sv[i] * rstd, acc[c + i * E]);
                d[i] = fmaf(rstd, g[i] * gy[i] - sv[i] * m, d[i]);
            }
            if (dx) store_n<kE, VEC, kStep<VEC>>(dx + row * D + c, d, D - c);
            if (dres) store_n<kE, VEC, kStep<VEC>>(dres + row * D + c, d, D - c);
        }
    }
    for (int c = first; c < D; c += step)
#pragma unroll
        for (int i = 0; i < kE; ++i)
            if (c + i * E < D) part[(size_t)blockIdx.x * D + c + i * E] = acc[c + i * E];
}

// Vectors per thread: the fewest that fit 512 threads, but two from 4096 channels on (16384 x 4096
// with a bf16 residual: 84 us for 110 with one, gradient 89 for 110).  Two would pay from 2048
// channels on as well: 16384 rows take 41 us for the 47 of one, gradient 49 for 55.
int norm_vpt(int D) { return D < 4096 ? 1 : D <= 8192 ? 2 : D <= 16384 ? 4 : 8; }
// The gradient's rows past this are wide (8192 x 8192 in registers 91 us, as wide rows 264).
constexpr int kWide = 8192;
constexpr int kWidest = 32768;   // channels that the entry points accept
template <typename TIn, typename TRes, int EIGHT, int VPT>
void norm_run(const AddNormArgs &a, bool vec, cudaStream_t st)
{
    const int nt = norm_threads(a.D, VPT);
    const dim3 grid((unsigned)std::min<long long>(a.rows, 152LL * std::max(1, norm_threads_sm(EIGHT) / nt))), block(nt);
    if (vec)
        add_rmsnorm_kernel<TIn, TRes, EIGHT, VPT, true><<<grid, block, 0, st>>>(
            (const TIn *)a.x, (const TRes *)a.residual, a.weight, a.y, a.scale, (TRes *)a.residual_out, a.rows, a.D,
            a.eps);
    else
        add_rmsnorm_kernel<TIn, TRes, EIGHT, VPT, false><<<grid, block, 0, st>>>(
            (const TIn *)a.x, (const TRes *)a.residual, a.weight, a.y, a.scale, (TRes *)a.residual_out, a.rows, a.D,
            a.eps);
}

template <typename TIn, typename TRes>
void norm_pick(const AddNormArgs &a, bool vec, cudaStream_t st)
{
    const int v = norm_vpt(a.D);
    const int e = !a.scale ? 0 : a.group ? 2 : 1;
#define LDN_NORM(E, V) norm_run<TIn, TRes, E, V>(a, vec, st)
    if (e == 0) v == 1 ? LDN_NORM(0, 1) : v == 2 ? LDN_NORM(0, 2) : v == 4 ? LDN_NORM(0, 4) : LDN_NORM(0, 8);
    if (e == 1) v == 1 ? LDN_NORM(1, 1) : v == 2 ? LDN_NORM(1, 2) : v == 4 ? LDN_NORM(1, 4) : LDN_NORM(1, 8);
    if (e == 2) v == 1 ? LDN_NORM(2, 1) : v == 2 ? LDN_NORM(2, 2) : v == 4 ? LDN_NORM(2, 4) : LDN_NORM(2, 8);
#undef LDN_NORM
}

template <typename TIn, typename TRes, int VPT>
void norm_bwd_run(const AddNormBwdArgs &a, int grid, bool vec, cudaStream_t st)
{
    const dim3 block(norm_threads(a.D, VPT));
    if (vec)
        add_rmsnorm_bwd_kernel<TIn, TRes, VPT, true><<<grid, block, 0, st>>>(
            (const TIn *)a.dy, (const TRes *)a.s, a.weight, (const TRes *)a.dsum, (TIn *)a.dx, (TRes *)a.dres,
            a.part, a.rows, a.D, a.eps);
    else
        add_rmsnorm_bwd_kernel<TIn, TRes, VPT, false><<<grid, block, 0, st>>>(
            (const TIn *)a.dy, (const TRes *)a.s, a.weight, (const TRes *)a.dsum, (TIn *)a.dx, (TRes *)a.dres,
            a.part, a.rows, a.D, a.eps);
}

template <typename TIn, typename TRes, bool VEC>
cudaError_t norm_bwd_wide(const AddNormBwdArgs &a, int grid, cudaStream_t st)
{
    auto *k = add_rmsnorm_bwd_wide_kernel<TIn, TRes, VEC>;
    // the attribute is the kernel's, shared by all host threads: always the widest row's, so that a
    // call between another's two lines changes nothing
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kWidest * (int)sizeof(float));
    if (e != cudaSuccess) return e;
    k<<<grid, kMostThreads, a.D * sizeof(float), st>>>((const TIn *)a.dy, (const TRes *)a.s, a.weight,
                                                       (const TRes *)a.dsum, (TIn *)a.dx, (TRes *)a.dres, a.part,
                                                       a.rows, a.D, a.eps);
    return cudaGetLastError();
}

template <typename TIn, typename TRes>
cudaError_t norm_bwd_pick(const AddNormBwdArgs &a, int grid, bool vec, cudaStream_t st)
{
    if (a.D > kWide)
        return vec ? norm_bwd_wide<TIn, TRes, true>(a, grid, st) : norm_bwd_wide<TIn, TRes, false>(a, grid, st);
    if (norm_vpt(a.D) == 1) norm_bwd_run<TIn, TRes, 1>(a, grid, vec, st);
    else norm_bwd_run<TIn, TRes, 2>(a, grid, vec, st);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_add_rmsnorm(const AddNormArgs &a, cudaStream_t st)
{
    const bool vec = a.D % kE == 0 && vec16(a.x) && vec16(a.residual) && vec16(a.residual_out) &&
                     vec16(a.weight) && (a.scale ? ((uintptr_t)a.y & 7u) == 0 : vec16(a.y));
    if (a.dtype == LDN_F32) norm_pick<float, float>(a, vec, st);
    else if (a.res_dtype == LDN_F32) norm_pick<__nv_bfloat16, float>(a, vec, st);
    else norm_pick<__nv_bfloat16, __nv_bfloat16>(a, vec, st);
    return cudaGetLastError();
}

// Blocks of the gradient's row walk: 512 threads an SM (one block of wide rows), no more than
// rows: two 256-thread blocks an SM with the next row on its way keep HBM busy, and each block
// more is a row more for the column sum (8192 x 2048, with one row on its way: 54 us at 512
// threads, 57 at 1024, 64 at 2048, 81 at 256; two rows on their way take 2 us off).  A fixed
// 152 SMs, so that the workspace's size needs no device.
int add_rmsnorm_bwd_blocks(long long rows, int D)
{
    const int per = D > kWide ? 1 : std::max(1, 512 / norm_threads(D, norm_vpt(D)));
    return (int)std::min<long long>(rows, 152LL * per);
}

cudaError_t launch_add_rmsnorm_bwd(const AddNormBwdArgs &a, cudaStream_t st)
{
    const bool vec = a.D % kE == 0 && vec16(a.dy) && vec16(a.s) && vec16(a.dsum) && vec16(a.dx) && vec16(a.dres) &&
                     vec16(a.weight);
    const int grid = add_rmsnorm_bwd_blocks(a.rows, a.D);
    if (grid > 0) {
        const cudaError_t e = a.dtype == LDN_F32       ? norm_bwd_pick<float, float>(a, grid, vec, st)
                              : a.res_dtype == LDN_F32 ? norm_bwd_pick<__nv_bfloat16, float>(a, grid, vec, st)
                                                       : norm_bwd_pick<__nv_bfloat16, __nv_bfloat16>(a, grid, vec, st);
        if (e != cudaSuccess) return e;
    }
    column_sum_kernel<<<(a.D + 31) / 32, dim3(32, kSumRows), 0, st>>>(a.part, a.dweight, grid, a.D);
    return cudaGetLastError();
}

}  // namespace ldn
