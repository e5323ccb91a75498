#include "norm_residual_bwd.cuh"

namespace lsh {
template cudaError_t sub_bwd_type<__nv_bfloat16, false, false>(const SubCall&, const SubArgs&, const SubShape&,
                                                  cudaStream_t);
}  // namespace lsh
