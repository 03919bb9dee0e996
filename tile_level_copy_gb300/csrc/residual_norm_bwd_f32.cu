// Backward pass of the residual norm on rows of f32 (a file for each type, so that they compile side by side).
#include "residual_norm_bwd.cuh"

namespace moe {
template cudaError_t launch_residual_backward<float>(RnShape, const RnWeights&, const RnBackward&, int, bool, bool, int, cudaStream_t);
}
