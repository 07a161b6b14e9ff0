// The layer norm's kernels of rows of one type.
#include "norm_backward.cuh"
#include "norm_forward.cuh"

namespace nsk {

template cudaError_t norm_forward<float>(NormParams &, int, cudaStream_t);
template cudaError_t norm_backward<float>(NormParams &, int, cudaStream_t);

}  // namespace nsk
