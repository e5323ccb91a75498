#include "norm_residual_fwd.cuh"

namespace lsh {
template cudaError_t sub_fwd_type<float>(const SubCall&, const SubArgs&, const SubShape&, cudaStream_t);
}  // namespace lsh
