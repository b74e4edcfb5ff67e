#include "residual_kernels.cuh"

namespace mok {
namespace residual {
template cudaError_t forward_rows<float, float, true>(const ResidualParams&, cudaStream_t);
}  // namespace residual
}  // namespace mok
