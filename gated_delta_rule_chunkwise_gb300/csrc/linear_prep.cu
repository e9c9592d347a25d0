// What a product of the linear operators cannot take as it lies in memory is laid out first: rows that
// TMA cannot start at (16-byte boundaries), fp32 as planes of bf16, and dz of the gradients.
// Each moves its bytes once and is bound by HBM: dz of 8192 x 8192 with GELU and the bias's sums 62 us (6,500
// GB/s; 121 an element a thread, 73 with two rows of a warp on their way), fp32 777 x 1028 and 1001 x 1028 to
// planes 4 us.
#include "linear_common.cuh"
#include "sm100_ptx.cuh"

namespace ldn {
namespace linear {
namespace {

constexpr int kThreadsPrep = 256;

// Once in every kernel, before it touches memory.
__device__ __forceinline__ void begin()
{
    sm100::griddep_wait();
    sm100::griddep_launch_dependents();
}

template <typename T>
__global__ void __launch_bounds__(kThreadsPrep)
copy_rows_kernel(const T *__restrict__ src, long long ld, T *__restrict__ dst, long long ld_dst, long long rows, int width)
{
    begin();
    const int c = blockIdx.x * kThreadsPrep + threadIdx.x;
    if (c >= width) return;
    for (long long r = blockIdx.y; r < rows; r += gridDim.y) dst[r * ld_dst + c] = src[r * ld + c];
}

// x as the sum of three bf16 numbers, exactly (down to where the last falls below the smallest bf16):
// the nearest one to it, to what is left, and the rest.  What would round past the largest bf16 is cut
// off instead.  What is not finite is in the fourth plane alone, the one that only the largest parts'
// product reads: an infinity then meets no zero of the other operand's smaller planes.
struct Parts { float hi, mid, lo, all; };
__device__ __forceinline__ Parts parts(float x)
{
    const float size = fabsf(x);
    const bool finite = size <= 3.402823466e38f;
    const float v = finite ? x : 0.f;
    const float hi = size < 3.38e38f ? __bfloat162float(__float2bfloat16_rn(v))
                                     : __uint_as_float(__float_as_uint(v) & 0xffff0000u);
    const float mid = __bfloat162float(__float2bfloat16_rn(v - hi));
    return {hi, mid, v - hi - mid, finite ? hi : x};
}

// N neighbours of a row into its planes (N = 4, 8: as vectors).
template <int N> __device__ __forceinline__ void put_planes(const float *x, __nv_bfloat16 *p, long long plane)
{
    float v[4][N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const Parts q = parts(x[i]);
        v[0][i] = q.hi; v[1][i] = q.mid; v[2][i] = q.lo; v[3][i] = q.all;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) store_n<N, N != 1>(p + k * plane, v[k]);
}

// A block takes the rows that `rows_of` blocks share, 4 neighbours a thread where every row of src
// begins at a 16-byte boundary.
template <int N>
__global__ void __launch_bounds__(kThreadsPrep)
split_rows_kernel(const Split a, const Split b, int blocks_a)
{
    begin();
    const bool first = (int)blockIdx.y < blocks_a;
    const Split &s = first ? a : b;
    const int c = (blockIdx.x * kThreadsPrep + threadIdx.x) * N;
    const long long plane = s.ld_dst * s.rows;
    if (c >= s.width) return;
    for (long long r = first ? blockIdx.y : blockIdx.y - blocks_a; r < s.rows;
         r += first ? blocks_a : gridDim.y - blocks_a) {
        float v[N];
        load_n<N, N != 1>(s.src + r * s.ld + c, v);
        put_planes<N>(v, (__nv_bfloat16 *)s.dst + r * s.ld_dst + c, plane);
    }
}

// act'(z); FINE: of a z in fp32
template <bool FINE> __device__ __forceinline__ float2 slope(float2 z, int activation)
{
    if (activation == LDN_ACT_SILU) {   // g (1 + z (1 - g))
        const float2 g = rcp(__fadd2_rn(ex2(__fmul2_rn(z, dup(-kLog2e))), dup(1.f)));
        return __fmul2_rn(g, __ffma2_rn(z, __ffma2_rn(g, dup(-1.f), dup(1.f)), dup(1.f)));
    }
    float2 bell;   // Phi(z) + z phi(z)
    const float2 phi = normal_integral<FINE>(z, bell);
    return __ffma2_rn(__fmul2_rn(z, dup(0.39894228f)), bell, phi);
}

// dz = dy act'(z), as bf16 rows or planes of them, and each run of rows' share of its column sums.
// dz is rounded to bf16 for the tensor cores; the sums take it before.
// N neighbours a thread (8 where rows are whole vectors, 1 otherwise); a block takes 32 N columns and 8
// rows at a time, and adds the sums of its eight warps in a fixed order.
template <typename TY, typename TZ, bool PLANES, int N>
__global__ void __launch_bounds__(kThreadsPrep)
dz_kernel(const TY *__restrict__ dy, const TZ *__restrict__ z, __nv_bfloat16 *__restrict__ dz, long long ld_dz,
          long long plane, float *__restrict__ part, long long rows, int n, int activation, long long run)
{
    begin();
    constexpr int WARPS = kThreadsPrep / 32;
    constexpr bool VEC = N != 1;
    __shared__ float sm[WARPS][32 * N + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = (blockIdx.x * 32 + lane) * N;
    const long long r0 = blockIdx.y * run, r1 = min(rows, r0 + run);
    float sum[N];
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] = 0.f;
    constexpr int U = 4;   // rows of a warp on their way together
    if (c < n)
        for (long long r = r0 + warp; r < r1; r += U * WARPS) {
            Raw<TY, N, VEC> ry[U];
            Raw<TZ, N, VEC> rz[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const long long at = (r + u * WARPS) * n + c;
                const int valid = r + u * WARPS < r1 ? N : 0;
                ry[u].template load<VEC>(dy + at, valid);
                rz[u].template load<VEC>(z + at, z ? valid : 0);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const long long row = r + u * WARPS;
                if (row >= r1) break;
                float v[N];
                ry[u].widen(v);
                if (z) {
                    float q[N];
                    rz[u].widen(q);
#pragma unroll
                    for (int i = 0; i < N; i += 2) {
                        const float2 f = slope<sizeof(TZ) == 4>(make_float2(q[i], q[N == 1 ? i : i + 1]), activation);
                        v[i] *= f.x;
                        if (N > 1) v[N == 1 ? i : i + 1] *= f.y;
                    }
                }
#pragma unroll
                for (int i = 0; i < N; ++i) sum[i] += v[i];
                if (dz) {
                    if constexpr (PLANES) put_planes<N>(v, dz + row * ld_dz + c, plane);
                    else store_n<N, VEC>(dz + row * ld_dz + c, v);
                }
            }
        }
    if (!part) return;
#pragma unroll
    for (int i = 0; i < N; ++i) sm[warp][lane * N + i] = sum[i];
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * N; i += kThreadsPrep) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) t += sm[w][i];
        const int at = blockIdx.x * 32 * N + i;
        if (at < n) part[(long long)blockIdx.y * n + at] = t;
    }
}

constexpr int kSumRows = 32;
__global__ void __launch_bounds__(32 * kSumRows)
bias_sum_kernel(const float *__restrict__ part, void *__restrict__ out, int out_f32, int runs, int n)
{
    __shared__ float sm[kSumRows][33];
    begin();
    const int c = blockIdx.x * 32 + threadIdx.x, y = threadIdx.y;
    float t = 0.f;
    if (c < n)
        for (int i = y; i < runs; i += kSumRows) t += part[(long long)i * n + c];
    sm[y][threadIdx.x] = t;
    __syncthreads();
    if (y == 0 && c < n) {
#pragma unroll
        for (int i = 1; i < kSumRows; ++i) t += sm[i][threadIdx.x];
        if (out_f32) ((float *)out)[c] = t;
        else ((__nv_bfloat16 *)out)[c] = __float2bfloat16_rn(t);
    }
}

dim3 grid_for(long long rows, int width)
{
    return dim3((width + kThreadsPrep - 1) / kThreadsPrep, (unsigned)std::min<long long>(rows, 65535));
}

}  // namespace

cudaError_t copy_rows(const void *src, long long ld, void *dst, long long ld_dst, long long rows, int width, int bytes,
                      cudaStream_t st)
{
    const dim3 grid = grid_for(rows, width);
    if (bytes == 1)
        return launch_after(copy_rows_kernel<uint8_t>, grid, kThreadsPrep, 0, st, (const uint8_t *)src, ld, (uint8_t *)dst,
                            ld_dst, rows, width);
    return launch_after(copy_rows_kernel<uint16_t>, grid, kThreadsPrep, 0, st, (const uint16_t *)src, ld, (uint16_t *)dst,
                        ld_dst, rows, width);
}

cudaError_t split_rows(const Split &a, const Split &b, cudaStream_t st)
{
    auto vec = [](const Split &s) {
        return s.rows == 0 || (((uintptr_t)s.src & 15) == 0 && s.width % 4 == 0 && (s.ld % 4 == 0 || s.rows == 1));
    };
    const int n = vec(a) && vec(b) ? 4 : 1, widest = std::max(a.rows ? a.width : 1, b.rows ? b.width : 1);
    const int strips = (widest + kThreadsPrep * n - 1) / (kThreadsPrep * n);
    // a few rows a block, so that the card is full and no block ends at once
    auto blocks = [&](const Split &s) { return (int)std::min<long long>(s.rows, std::max(1, 152 * 16 / strips)); };
    const dim3 grid(strips, blocks(a) + blocks(b));
    return launch_after(n == 4 ? split_rows_kernel<4> : split_rows_kernel<1>, grid, kThreadsPrep, 0, st, a, b, blocks(a));
}

// Rows of a run, so that the blocks fill the card a few times and the sums' last step stays short.
static long long dz_run(long long rows, int n)
{
    const long long strips = (n + 255) / 256;   // of columns, of a vectored block
    const long long runs = std::max(1LL, std::min(256LL, 152 * 8 / strips));
    return std::max(32LL, (rows + runs - 1) / runs);
}
long long dz_runs(long long rows, int n) { return rows ? (rows + dz_run(rows, n) - 1) / dz_run(rows, n) : 0; }

template <typename TY, typename TZ, bool PLANES>
static cudaError_t run_dz(const void *dy, const void *z, __nv_bfloat16 *dz, long long ld_dz, long long plane, float *part,
                   long long rows, int n, int activation, cudaStream_t st)
{
    const long long run = dz_run(rows, n);
    const unsigned runs = (unsigned)dz_runs(rows, n);
    const bool vec = n % 8 == 0 && (((uintptr_t)dy | (uintptr_t)z) & 15) == 0;
    return launch_after(vec ? dz_kernel<TY, TZ, PLANES, 8> : dz_kernel<TY, TZ, PLANES, 1>,
                        dim3(vec ? (n + 255) / 256 : (n + 31) / 32, runs), kThreadsPrep, 0, st, (const TY *)dy,
                        (const TZ *)z, dz, ld_dz, plane, part, rows, n, activation, run);
}

cudaError_t form_dz(const void *dy, int dy_f32, const void *z, int activation, void *dz, long long ld_dz, long long plane,
                    bool planes, float *part, void *dbias, int bias_f32, long long rows, int n, cudaStream_t st)
{
    __nv_bfloat16 *d = (__nv_bfloat16 *)dz;
    const cudaError_t e =
        planes ? run_dz<float, float, true>(dy, z, d, ld_dz, plane, part, rows, n, activation, st)
        : dy_f32 ? run_dz<float, __nv_bfloat16, false>(dy, z, d, ld_dz, plane, part, rows, n, activation, st)
                 : run_dz<__nv_bfloat16, __nv_bfloat16, false>(dy, z, d, ld_dz, plane, part, rows, n, activation, st);
    if (e != cudaSuccess || !part) return e;
    return launch_after(bias_sum_kernel, dim3((n + 31) / 32), dim3(32, kSumRows), 0, st, part, dbias, bias_f32,
                        (int)dz_runs(rows, n), n);
}

}  // namespace linear
}  // namespace ldn
