// What the parts of the linear operators share.
#pragma once
#include "ldn_internal.cuh"
#include "mixer_common.cuh"

namespace ldn {
namespace linear {

// An operand: `planes` matrices of `rows` rows of `width`, as they lie in memory.
struct Operand {
    const void *p;
    long long width, rows, ld, plane;
    int planes;
};

struct Args {
    long long ni, nj;          // output: nj rows of ni
    int kblocks;               // of 128 bytes
    int chunk;                 // k blocks that are summed in tensor memory before they join the sum in registers
    int npairs;                // pairs of planes, four bits each: plane of A, plane of B
    uint32_t pairs_a, pairs_b;
    int bn, split, stages;     // the cut (linear_plan.h) and the stages of its ring
    // epilogue
    void *out, *z;             // [nj][ni]
    const void *bias, *residual;
    const float *scale_i, *scale_j;
    int out_f32, z_f32, bias_f32, activation;
    int staged;                // results leave through shared memory (linear_gemm.cuh)
    int *status;
};

// Phi(z), the normal distribution's integral, and phi(z) sqrt(2 pi) = e^(-z^2 / 2), from which both it
// and its slope come: the rational approximation 7.1.26 of Abramowitz and Stegun's handbook, within
// 0.8e-7 of Phi, and a few steps of fp32 at 1.
__device__ __forceinline__ float normal_integral(float z, float &bell)
{
    const float x = fabsf(z) * 0.70710678f;
    bell = ex2(-0.5f * kLog2e * (z * z));
    const float t = rcp(fmaf(0.3275911f, x, 1.f));
    float q = 1.061405429f;
    q = fmaf(q, t, -1.453152027f);
    q = fmaf(q, t, 1.421413741f);
    q = fmaf(q, t, -0.284496736f);
    q = fmaf(q, t, 0.254829592f);
    const float tail = 0.5f * (q * t) * bell;   // Phi(-|z|)
    return z > 0.f ? 1.f - tail : tail;         // NaN where z is
}

// Planes of an fp32 operand (split_rows): the largest part, the next, the last, and the largest with
// what is not finite.
constexpr int kPlanes = 4;

cudaError_t copy_rows(const void *src, long long ld, void *dst, long long ld_dst, long long rows, int width, int bytes,
                      cudaStream_t st);
// Rows of fp32 laid out as planes of bf16, of two operands in one launch (either may have no rows).
struct Split {
    const float *src;
    void *dst;
    long long ld, ld_dst, rows;   // a plane is ld_dst * rows elements
    int width;
};
cudaError_t split_rows(const Split &a, const Split &b, cudaStream_t st);
long long dz_runs(long long rows, int n);
// dz from dy and z (null: dz = dy), where dz is given; dbias, where part (dz_runs rows of n) is.
cudaError_t form_dz(const void *dy, int dy_f32, const void *z, int activation, void *dz, long long ld_dz, long long plane,
                    bool planes, float *part, void *dbias, int bias_f32, long long rows, int n, cudaStream_t st);

}  // namespace linear

cudaError_t linear_product(const linear::Operand &A, const linear::Operand &B, const linear::Args &a, cudaStream_t st);
cudaError_t linear_product_e4m3(const linear::Operand &A, const linear::Operand &B, const linear::Args &a,
                                cudaStream_t st);
cudaError_t linear_product_dx(const linear::Operand &A, const linear::Operand &B, const linear::Args &a, cudaStream_t st);
cudaError_t linear_product_dw(const linear::Operand &A, const linear::Operand &B, const linear::Args &a, cudaStream_t st);

}  // namespace ldn
