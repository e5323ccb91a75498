#include "norm_residual_fwd.cuh"

namespace lsh {
template cudaError_t sub_fwd_type<__nv_bfloat16>(const SubCall&, const SubArgs&, const SubShape&, cudaStream_t);
}  // namespace lsh
