// Forward pass of the residual norm on rows of f16 (a file for each type, so that they compile side by side).
#include "residual_norm_fwd.cuh"

namespace moe {
template cudaError_t launch_residual_forward<__half>(RnShape, const RnWeights&, const RnForward&, int, int, cudaStream_t);
}
