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
    int split;
    // epilogue
    void *out, *z;             // [nj][ni]
    const void *bias, *residual;
    const float *scale_i, *scale_j;
    int out_f32, z_f32, bias_f32, activation;
    int *status;
};

// Planes of an fp32 operand (split_rows): the largest part, the next, the last, and the largest with
// what is not finite.
constexpr int kPlanes = 4;

cudaError_t copy_rows(const void *src, long long ld, void *dst, long long ld_dst, long long rows, int width, int bytes,
                      cudaStream_t st);
cudaError_t split_rows(const float *src, long long ld, void *dst, long long ld_dst, long long plane, long long rows,
                       int width, cudaStream_t st);
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
