// Shapes and values that the passes of the residual norm share.
#pragma once

#include "row_values.cuh"

namespace moe {

constexpr int RN_MAX_D = 16384;

// How a launch's threads share the rows: groups of `warps` warps, `groups` of them in a CTA; a thread holds up to
// `pieces` pieces of each row in every one of `slots` slots of shared memory.
struct RnShape {
    int64_t rows, gate_rows;  // gate_rows 0: no gate
    int64_t chunk;            // backward: consecutive rows of a group of warps
    int d, warps, groups, pieces, slots;
    int post, pre;            // MOE_NORM_*
    float eps, inv_d, res, branch;
};
// form: how the vectors that are there lie, LN_W_*.
struct RnWeights {
    const void *post_w, *post_b, *gate, *pre_w, *pre_b;
    int form;
    bool f32;
};
struct RnBackward {
    const void *dz, *dh, *u, *h;
    const float2 *post_stats, *pre_stats;
    void *dx, *du;
    float* part;   // the CTAs' sums
    float* gpart;  // [groups of warps][2][d]: sums of the gates whose rows lie in more than one group of warps
    float* gsum;   // [groups of warps][2][d], with more than one gate: sums of post_w's and post_b's gradients so far
    void* dgate;
};

// Launches the backward kernel on rows of T (one file for each type).
template <typename T>
cudaError_t launch_residual_backward(const RnShape& s, const RnWeights& w, const RnBackward& b, int vec, bool full,
                                     bool grouped, int ctas, cudaStream_t st);

// Backward: values of a thread (32 of them spill; only rows above 8192 need them).
inline int rn_backward_values(int d) { return d <= 8192 ? 16 : 32; }

namespace {

// VEC weights from column c on (null: `none`).
template <typename T, int VEC>
__device__ __forceinline__ void weight(const RnWeights& w, const void* p, float none, int64_t c,
                                       typename Lanes<VEC>::V (&o)[Lanes<VEC>::N]) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < Lanes<VEC>::N; ++i) o[i] = both<typename Lanes<VEC>::V>(none);
        return;
    }
    if (w.form == LN_W_F32) weights<T, VEC, LN_W_F32>(static_cast<const float*>(p) + c, true, none, 0, o);
    else if (w.form == LN_W_SAME) weights<T, VEC, LN_W_SAME>(static_cast<const T*>(p) + c, false, none, 0, o);
    else if (w.f32) weights<T, VEC, LN_W_ANY>(static_cast<const float*>(p) + c, true, none, 0, o);
    else weights<T, VEC, LN_W_ANY>(static_cast<const T*>(p) + c, false, none, 0, o);
}

template <typename T>
__device__ __forceinline__ float value_at(const void* p, bool f32, int64_t i, float none) {
    return !p ? none : f32 ? static_cast<const float*>(p)[i] : num(static_cast<const T*>(p)[i]);
}
template <typename P>
__device__ __forceinline__ void fetch(P* to, const P* from) {  // asynchronous where the piece allows it
    if constexpr (sizeof(P) >= 4) copy_async<sizeof(P)>(to, from);
    else *to = *from;
}
__device__ __forceinline__ void fetched(int pending) {  // all but the last `pending` groups are there
    if (pending == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (pending == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 2;" ::: "memory");
}

}  // namespace
}  // namespace moe
