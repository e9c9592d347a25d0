// What a product of the linear operators cannot take as it lies in memory is laid out first: rows that
// TMA cannot start at (16-byte boundaries), fp32 as planes of bf16, and dz of the gradients.
// Each moves its bytes once and is bound by HBM.
#include "linear_common.cuh"

namespace ldn {
namespace linear {
namespace {

constexpr int kThreadsPrep = 256;

template <typename T>
__global__ void __launch_bounds__(kThreadsPrep)
copy_rows_kernel(const T *__restrict__ src, long long ld, T *__restrict__ dst, long long ld_dst, long long rows, int width)
{
    const int c = blockIdx.x * kThreadsPrep + threadIdx.x;
    if (c >= width) return;
    for (long long r = blockIdx.y; r < rows; r += gridDim.y) dst[r * ld_dst + c] = src[r * ld + c];
}

// x as the sum of three bf16 numbers, exactly (down to where the last falls below the smallest bf16):
// the nearest one to it, to what is left, and the rest.  What would round past the largest bf16 is cut
// off instead.  What is not finite is in the fourth plane alone, the one that only the largest parts'
// product reads: an infinity then meets no zero of the other operand's smaller planes.
__device__ __forceinline__ void split_f32(float x, __nv_bfloat16 *p, long long plane)
{
    const float size = fabsf(x);
    const bool finite = size <= 3.402823466e38f;
    const float v = finite ? x : 0.f;
    const float hi = size < 3.38e38f ? __bfloat162float(__float2bfloat16_rn(v))
                                     : __uint_as_float(__float_as_uint(v) & 0xffff0000u);
    const float mid = __bfloat162float(__float2bfloat16_rn(v - hi));
    p[0] = __float2bfloat16_rn(hi);
    p[plane] = __float2bfloat16_rn(mid);
    p[2 * plane] = __float2bfloat16_rn(v - hi - mid);
    p[3 * plane] = __float2bfloat16_rn(finite ? hi : x);
}

__global__ void __launch_bounds__(kThreadsPrep)
split_rows_kernel(const float *__restrict__ src, long long ld, __nv_bfloat16 *__restrict__ dst, long long ld_dst,
                  long long plane, long long rows, int width)
{
    const int c = blockIdx.x * kThreadsPrep + threadIdx.x;
    if (c >= width) return;
    for (long long r = blockIdx.y; r < rows; r += gridDim.y) split_f32(src[r * ld + c], dst + r * ld_dst + c, plane);
}

// act'(z)
__device__ __forceinline__ float slope(float z, int activation)
{
    if (activation == LDN_ACT_SILU) {
        const float g = sigmoid_fast(z);
        return g * fmaf(z, 1.f - g, 1.f);
    }
    // Phi(z) + z phi(z)
    return fmaf(0.5f, erff(z * 0.70710678f), 0.5f) + z * 0.39894228f * ex2(-0.5f * kLog2e * z * z);
}

// dz = dy act'(z), as bf16 rows or planes of them, and each run of rows' share of its column sums.
// dz is rounded to bf16 for the tensor cores; the sums take it before.
template <typename TY, typename TZ, bool PLANES>
__global__ void __launch_bounds__(kThreadsPrep)
dz_kernel(const TY *__restrict__ dy, const TZ *__restrict__ z, __nv_bfloat16 *__restrict__ dz, long long ld_dz,
          long long plane, float *__restrict__ part, long long rows, int n, int activation, long long run)
{
    const int c = blockIdx.x * kThreadsPrep + threadIdx.x;
    if (c >= n) return;
    const long long r0 = blockIdx.y * run, r1 = min(rows, r0 + run);
    float sum = 0.f;
#pragma unroll 4
    for (long long r = r0; r < r1; ++r) {
        float v = (float)dy[r * n + c];
        if (z) v *= slope((float)z[r * n + c], activation);
        sum += v;
        if (dz) {
            if constexpr (PLANES) split_f32(v, dz + r * ld_dz + c, plane);
            else dz[r * ld_dz + c] = __float2bfloat16_rn(v);
        }
    }
    if (part) part[(long long)blockIdx.y * n + c] = sum;
}

constexpr int kSumRows = 32;
__global__ void __launch_bounds__(32 * kSumRows)
bias_sum_kernel(const float *__restrict__ part, void *__restrict__ out, int out_f32, int runs, int n)
{
    __shared__ float sm[kSumRows][33];
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
    if (bytes == 1)
        copy_rows_kernel<<<grid_for(rows, width), kThreadsPrep, 0, st>>>((const uint8_t *)src, ld, (uint8_t *)dst, ld_dst,
                                                                         rows, width);
    else
        copy_rows_kernel<<<grid_for(rows, width), kThreadsPrep, 0, st>>>((const uint16_t *)src, ld, (uint16_t *)dst,
                                                                         ld_dst, rows, width);
    return cudaGetLastError();
}

cudaError_t split_rows(const float *src, long long ld, void *dst, long long ld_dst, long long plane, long long rows,
                       int width, cudaStream_t st)
{
    split_rows_kernel<<<grid_for(rows, width), kThreadsPrep, 0, st>>>(src, ld, (__nv_bfloat16 *)dst, ld_dst, plane, rows,
                                                                      width);
    return cudaGetLastError();
}

// Rows of a run, so that the blocks fill the card a few times and the sums' last step stays short.
static long long dz_run(long long rows, int n)
{
    const long long strips = (n + kThreadsPrep - 1) / kThreadsPrep;
    const long long runs = std::max(1LL, std::min(1024LL, 152 * 8 / strips));
    return std::max(8LL, (rows + runs - 1) / runs);
}
long long dz_runs(long long rows, int n) { return rows ? (rows + dz_run(rows, n) - 1) / dz_run(rows, n) : 0; }

cudaError_t form_dz(const void *dy, int dy_f32, const void *z, int activation, void *dz, long long ld_dz, long long plane,
                    bool planes, float *part, void *dbias, int bias_f32, long long rows, int n, cudaStream_t st)
{
    const int runs = (int)dz_runs(rows, n);
    const long long run = dz_run(rows, n);
    const dim3 grid((n + kThreadsPrep - 1) / kThreadsPrep, runs);
    __nv_bfloat16 *d = (__nv_bfloat16 *)dz;
    if (planes)
        dz_kernel<float, float, true><<<grid, kThreadsPrep, 0, st>>>((const float *)dy, (const float *)z, d, ld_dz, plane,
                                                                     part, rows, n, activation, run);
    else if (dy_f32)
        dz_kernel<float, __nv_bfloat16, false><<<grid, kThreadsPrep, 0, st>>>(
            (const float *)dy, (const __nv_bfloat16 *)z, d, ld_dz, plane, part, rows, n, activation, run);
    else
        dz_kernel<__nv_bfloat16, __nv_bfloat16, false><<<grid, kThreadsPrep, 0, st>>>(
            (const __nv_bfloat16 *)dy, (const __nv_bfloat16 *)z, d, ld_dz, plane, part, rows, n, activation, run);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !part) return e;
    bias_sum_kernel<<<(n + 31) / 32, dim3(32, kSumRows), 0, st>>>(part, dbias, bias_f32, runs, n);
    return cudaGetLastError();
}

}  // namespace linear
}  // namespace ldn
