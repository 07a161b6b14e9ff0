// The layer norm's kernels of rows of one type.
#include "norm_backward.cuh"
#include "norm_forward.cuh"

namespace nsk {

template cudaError_t norm_forward<__nv_bfloat16>(NormParams &, int, cudaStream_t);
template cudaError_t norm_backward<__nv_bfloat16>(NormParams &, int, cudaStream_t);

}  // namespace nsk
