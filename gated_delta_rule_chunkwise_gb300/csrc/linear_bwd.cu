// Products of the gradients: dx, with the weight's rows as k, and dweight, with the tokens as k.
#include "linear_launch.cuh"

namespace ldn {
cudaError_t linear_product_dx(const linear::Operand &A, const linear::Operand &B, const linear::Args &a,
                              cudaStream_t st)
{
    return linear::run<true, false, false, false>(A, B, a, st);
}
cudaError_t linear_product_dw(const linear::Operand &A, const linear::Operand &B, const linear::Args &a,
                              cudaStream_t st)
{
    return linear::run<true, true, false, false>(A, B, a, st);
}
}  // namespace ldn
