// Products of the forward: both operands as rows of k.
#include "linear_launch.cuh"

namespace ldn {
cudaError_t linear_product(const linear::Operand &A, const linear::Operand &B, const linear::Args &a, cudaStream_t st)
{
    return linear::run<false, false, false, true>(A, B, a, st);
}
}  // namespace ldn
