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

// Phi(z), the normal distribution's integral, and e^(-z^2 / 2), from which both it and its slope come, of
// two values in packed arithmetic.  The tail Phi(-|z|) is e^(-z^2 / 2) t P(t) with t = 1 / (1 + p |z|): its
// quotient by the exponential falls like 1 / |z|, which t does too.
// FINE: p = 0.34 and P of degree 8, of the least largest relative error up to |z| = 13.3, where the tail leaves
// fp32 (reweighted least squares over Chebyshev polynomials): 2.5e-8.  With fp32's roundings Phi is within 5e-7 of
// itself down to z = -2, and below that within what the exponential's rounded argument leaves (2e-6 at -6);
// 0.5 (1 + erf) in fp32 has 9e-7 at -2 and no digit at -6.
// Otherwise 7.1.26 of Abramowitz and Stegun's handbook (coefficients halved: the tail of Phi is half of erfc's),
// within 2.6e-7 of Phi: for slopes at a z of 8 bits, whose other term outgrows what is left of Phi far out (dz of
// 8192 x 8192 62 us, 69 with the finer one).
template <bool FINE> __device__ __forceinline__ float2 normal_integral(float2 z, float2 &bell)
{
    constexpr float fine[] = {0.135618857f, 0.13614239f,  0.114967484f, 0.116314463f, -0.0470853787f,
                              0.205778794f, -0.276415287f, 0.141150721f, -0.0264720305f};
    constexpr float plain[] = {0.5f * 0.254829592f, 0.5f * -0.284496736f, 0.5f * 1.421413741f, 0.5f * -1.453152027f,
                               0.5f * 1.061405429f};
    constexpr int DEGREE = FINE ? 8 : 4;
    bell = ex2(__fmul2_rn(__fmul2_rn(z, z), dup(-0.5f * kLog2e)));
    const float2 t = rcp(__ffma2_rn(make_float2(fabsf(z.x), fabsf(z.y)), dup(FINE ? 0.34f : 0.3275911f * 0.70710678f),
                                    dup(1.f)));
    float2 q = dup(FINE ? fine[8] : plain[4]);
#pragma unroll
    for (int i = DEGREE; i-- > 0;) q = __ffma2_rn(q, t, dup(FINE ? fine[i] : plain[i]));
    const float2 tail = __fmul2_rn(__fmul2_rn(q, t), bell);   // Phi(-|z|); NaN where z is
    return make_float2(z.x > 0.f ? 1.f - tail.x : tail.x, z.y > 0.f ? 1.f - tail.y : tail.y);
}
__device__ __forceinline__ float2 gelu(float2 z)
{
    float2 bell;
    return __fmul2_rn(z, normal_integral<true>(z, bell));
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
