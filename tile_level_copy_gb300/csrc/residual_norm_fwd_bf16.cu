// Forward pass of the residual norm on rows of bf16 (a file for each type, so that they compile side by side).
#include "residual_norm_fwd.cuh"

namespace moe {
template cudaError_t launch_residual_forward<__nv_bfloat16>(RnShape, const RnWeights&, const RnForward&, int, int, cudaStream_t);
}
