// Backward pass of the residual norm on rows of bf16 (a file for each type, so that they compile side by side).
#include "residual_norm_bwd.cuh"

namespace moe {
template cudaError_t launch_residual_backward<__nv_bfloat16>(RnShape, const RnWeights&, const RnBackward&, int, bool, bool, int, cudaStream_t);
}
