// Products of the forward in 8 bits: both operands as rows of k in e4m3.
#include "linear_launch.cuh"

namespace ldn {
cudaError_t linear_product_e4m3(const linear::Operand &A, const linear::Operand &B, const linear::Args &a,
                                cudaStream_t st)
{
    return linear::run<false, false, true, true>(A, B, a, st);
}
}  // namespace ldn
