#include "residual_kernels.cuh"

namespace mok {
namespace residual {
template cudaError_t backward_rows<__nv_bfloat16, __nv_bfloat16, false>(const ResidualParams&, int*, cudaStream_t);
}  // namespace residual
}  // namespace mok
