#include "norm_residual_bwd.cuh"

namespace lsh {
template cudaError_t sub_bwd_type<float, false, true>(const SubCall&, const SubArgs&, const SubShape&,
                                                  cudaStream_t);
}  // namespace lsh
