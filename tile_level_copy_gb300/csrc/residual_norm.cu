// Norms around a block fused with its gate and the residual sum: the C entries, and the sums over the rows that end the
// backward pass.
#include "residual_norm.cuh"

#include <math.h>

#include <initializer_list>

namespace moe {
namespace {

constexpr int RN_RED_COLS = 32, RN_RED_ROWS = 32, RN_RED_FLY = 10;
constexpr int RN_MAX_SMS = 256;

// The gradients of the weights from the CTAs' sums [parts][sums][d]: blockIdx.y 0 the norm before the next block
// (sum 0, and 1 with full), 1 the norm behind this one and a gate that all rows share (the last one or two sums).
// blockIdx.y from 2 on: the gradients of the gates whose rows lie in more than one group of warps.
struct RnReduce {
    const float* part;
    const float* gpart;
    int parts, d;
    bool full, grouped, f32;
    const void *post_w, *post_b, *gate;
    void *dpost_w, *dpost_b, *dgate, *dpre_w, *dpre_b;
    int64_t rows, gate_rows, chunk;
    int64_t shared;  // gates, or places between groups of warps, whichever are fewer
    bool at_places;
    int each;  // warps for one of them, a power of two: four rows of sums in flight each
};
template <typename T>
__device__ __forceinline__ void put_at(void* p, bool f32, int64_t i, float v) {
    if (!p) return;
    if (f32) static_cast<float*>(p)[i] = v;
    else put(static_cast<T*>(p)[i], v);
}
__device__ __forceinline__ int64_t over(int64_t a, int64_t b) {  // (a quotient of 64 bits takes four times as long)
    return (uint64_t)(a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}
// These gates' gradients from the groups' sums, as many at once as a CTA's warps do. The gates are found among all or, where these
// are more, among the places where one group's rows end and the next one's begin: at row b chunk; a gate that lies
// around several such places is that of the first. (With a gate for each of 16384 rows most need nothing: going over them
// took 600 us.)
template <typename T>
__device__ __forceinline__ void shared_gates(const RnReduce& a, float (*acc)[RN_RED_COLS], int lane, int row, int c) {
    const int each = a.each, gates = RN_RED_ROWS / each, mine = row / each, first = row % each;
    for (int64_t i0 = (int64_t)(blockIdx.y - 2) * gates; i0 < a.shared; i0 += (int64_t)(gridDim.y - 2) * gates) {
        const int64_t i = i0 + mine;
        int64_t g = 0, from = 0, w0 = 0, w1 = 0;
        bool there = i < a.shared;
        if (there) {
            g = a.at_places ? over((i + 1) * a.chunk, a.gate_rows) : i;
            from = g * a.gate_rows;
            const int64_t to = from + a.gate_rows < a.rows ? from + a.gate_rows : a.rows;
            if (a.at_places) there = from < (i + 1) * a.chunk && from >= i * a.chunk;
            w0 = a.at_places ? i : over(from, a.chunk);
            w1 = over(to - 1, a.chunk);
            there = there && w0 < w1;  // (else the group of warps wrote it)
        }
        float v = 0.f;
        if (there && c < a.d) {  // only the first group of warps may have begun with an earlier gate
            for (int64_t k = w0 + first; k <= w1; k += 4 * each) {  // four loads in flight
                float e[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int64_t at = k + n * each;
                    e[n] = at <= w1 ? a.gpart[(2 * at + (at == w0 && w0 * a.chunk < from ? 1 : 0)) * a.d + c] : 0.f;
                }
#pragma unroll
                for (int n = 0; n < 4; ++n) v += e[n];
            }
        }
        if (!__syncthreads_or(there)) continue;
        acc[row][lane] = v;
        __syncthreads();
        if (there && first == 0 && c < a.d) {
            for (int q = 1; q < each; ++q) v += acc[row + q][lane];
            put_at<T>(a.dgate, a.f32, g * a.d + c, v);
        }
    }
}
template <typename T>
__global__ void __launch_bounds__(RN_RED_COLS* RN_RED_ROWS) rn_reduce_kernel(RnReduce a) {
    __shared__ float acc[2][RN_RED_ROWS][RN_RED_COLS];
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x % RN_RED_COLS, row = threadIdx.x / RN_RED_COLS, c = blockIdx.x * RN_RED_COLS + lane;
    if (blockIdx.y >= 2) {
        shared_gates<T>(a, acc[0], lane, row, c);
        return;
    }
    const int sums = a.full ? 4 : 2, first = blockIdx.y == 0 ? 0 : sums / 2;
    float v[2] = {0.f, 0.f};
    if (c < a.d) {
        const float* const from = a.part + (size_t)first * a.d + c;
        const size_t hop = (size_t)sums * a.d;
        const int second = a.full ? a.d : 0;
        for (int q = row; q < a.parts; q += RN_RED_FLY * RN_RED_ROWS) {  // all loads of both sums in flight
            float e[RN_RED_FLY], f[RN_RED_FLY];
#pragma unroll
            for (int k = 0; k < RN_RED_FLY; ++k) {
                const bool there = q + k * RN_RED_ROWS < a.parts;
                const float* const p = from + (size_t)(q + k * RN_RED_ROWS) * hop;
                e[k] = there ? *p : 0.f;
                f[k] = there && a.full ? p[second] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < RN_RED_FLY; ++k) {
                v[0] += e[k];
                v[1] += f[k];
            }
        }
    }
    acc[0][row][lane] = v[0];
    acc[1][row][lane] = v[1];
    __syncthreads();
    if (row || c >= a.d) return;
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int q = 0; q < RN_RED_ROWS; ++q) {
        x += acc[0][q][lane];
        y += acc[1][q][lane];
    }
    if (blockIdx.y == 0) {
        put_at<T>(a.dpre_w, a.f32, c, x);
        put_at<T>(a.dpre_b, a.f32, c, y);
    } else if (a.grouped) {
        put_at<T>(a.dpost_w, a.f32, c, x);
        put_at<T>(a.dpost_b, a.f32, c, y);
    } else {  // the sums lack the gate's factor
        const float g = value_at<T>(a.gate, a.f32, c, 1.f);
        put_at<T>(a.dpost_w, a.f32, c, x * g);
        put_at<T>(a.dpost_b, a.f32, c, y * g);
        put_at<T>(a.dgate, a.f32, c, value_at<T>(a.post_w, a.f32, c, 1.f) * x + value_at<T>(a.post_b, a.f32, c, 0.f) * y);
    }
}

int check(const moe_residual_norm_config* c) {
    if (!c) return fail(MOE_ERR_ARG, "config is NULL");
    if (c->rows < 0 || c->gate_rows < 0)
        return fail(MOE_ERR_ARG, "rows=%lld and gate_rows=%lld must be >= 0", (long long)c->rows, (long long)c->gate_rows);
    if (c->d < 1 || c->d > RN_MAX_D) return fail(MOE_ERR_ARG, "d=%d must be in [1, %d]", c->d, RN_MAX_D);
    if (c->rows > INT64_MAX / 8 / c->d || c->rows > INT64_C(1) << 38) return fail(MOE_ERR_ARG, "rows=%lld is too large", (long long)c->rows);
    if (c->dtype != MOE_DTYPE_F32 && c->dtype != MOE_DTYPE_BF16 && c->dtype != MOE_DTYPE_F16)
        return fail(MOE_ERR_ARG, "dtype=%d is not a MOE_DTYPE", c->dtype);
    if (c->wdtype != MOE_DTYPE_F32 && c->wdtype != c->dtype)
        return fail(MOE_ERR_ARG, "wdtype=%d must be fp32 or dtype", c->wdtype);
    for (int k : {c->post, c->pre})
        if (k != MOE_NORM_NONE && k != MOE_NORM_RMS && k != MOE_NORM_LAYER)
            return fail(MOE_ERR_ARG, "post=%d and pre=%d must be MOE_NORM_*", c->post, c->pre);
    if (!(c->eps >= 0)) return fail(MOE_ERR_ARG, "eps=%g must be >= 0", (double)c->eps);
    if (!isfinite(c->residual_scale) || !isfinite(c->branch_scale))
        return fail(MOE_ERR_ARG, "residual_scale=%g and branch_scale=%g must be finite", (double)c->residual_scale,
                    (double)c->branch_scale);
    for (int i = 0; i < 4; ++i)
        if (c->reserved[i]) return fail(MOE_ERR_ARG, "reserved fields must be zero");
    return MOE_OK;
}

// Whether rows of outputs lie over one another or over rows that they may not: an output may be an input that its
// elements replace one by one (the same pointer), and nothing else of it.
struct Span {
    const void* p;
    size_t bytes;
};
bool apart(const Span& a, const Span& b) {
    if (!a.p || !b.p) return true;
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.p), q = reinterpret_cast<uintptr_t>(b.p);
    return p >= q + b.bytes || q >= p + a.bytes;
}
bool apart_or_same(const void* a, const void* b, size_t bytes) { return a == b || apart({a, bytes}, {b, bytes}); }
// Every output lies apart from these inputs and from the outputs behind it in the list. (Weights, gates and statistics are read
// while other rows' outputs are written, in the forward pass by loads that no store may change.)
int check_apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (const Span* o = outs.begin(); o != outs.end(); ++o) {
        if (!o->p) continue;
        for (const Span* i = o + 1; i != outs.end(); ++i)
            if (!apart(*o, *i)) return fail(MOE_ERR_ARG, "two outputs share memory");
        for (const Span& i : ins)
            if (!apart(*o, i)) return fail(MOE_ERR_ARG, "an output shares memory with a weight, a gate, statistics or the workspace");
    }
    return MOE_OK;
}
size_t gate_bytes(const moe_residual_norm_config& c) {
    return c.gate_rows > 0 ? (size_t)((c.rows - 1) / c.gate_rows + 1) * c.d * dtype_size(c.wdtype) : 0;
}

// 16-byte pieces where they divide the rows and every row's pieces are aligned, else single values.
template <typename... Ptr>
int vector_width(const moe_residual_norm_config& c, Ptr... p) {
    const int v = (int)(16 / dtype_size(c.dtype));
    return c.d % v == 0 && (aligned(p, 16) && ...) ? v : 1;
}
RnWeights weights_of(const moe_residual_norm_config& c, const void* post_w, const void* post_b, const void* gate,
                     const void* pre_w, const void* pre_b) {
    const bool whole = aligned(post_w, 16) && aligned(post_b, 16) && aligned(gate, 16) && aligned(pre_w, 16) && aligned(pre_b, 16);
    return RnWeights{post_w, post_b, gate, pre_w, pre_b, c.wdtype == MOE_DTYPE_F32, whole};
}
int check_weights(const moe_residual_norm_config& c, const void* post_w, const void* post_b, const void* gate,
                  const void* pre_w, const void* pre_b) {
    const size_t we = dtype_size(c.wdtype);
    if (!aligned(post_w, we) || !aligned(post_b, we) || !aligned(gate, we) || !aligned(pre_w, we) || !aligned(pre_b, we))
        return fail(MOE_ERR_ARG, "a weight is not aligned to its type");
    if ((post_b && c.post != MOE_NORM_LAYER) || (pre_b && c.pre != MOE_NORM_LAYER))
        return fail(MOE_ERR_ARG, "a bias goes with MOE_NORM_LAYER");
    if ((post_w && !c.post) || (pre_w && !c.pre)) return fail(MOE_ERR_ARG, "a weight without its norm");
    if (c.rows > 0 && (gate != nullptr) != (c.gate_rows > 0)) return fail(MOE_ERR_ARG, "gate goes with gate_rows=%lld", (long long)c.gate_rows);
    return MOE_OK;
}

RnShape shape_of(const moe_residual_norm_config& c) {
    RnShape s;
    s.rows = c.rows;
    s.gate_rows = c.gate_rows < c.rows ? c.gate_rows : c.rows;  // of one gate for all rows, as many as there are
    s.chunk = 0;
    s.d = c.d;
    s.warps = s.groups = s.slots = 1;
    s.post = c.post, s.pre = c.pre;
    s.eps = c.eps;
    s.inv_d = 1.0f / (float)c.d;
    s.res = c.residual_scale, s.branch = c.branch_scale;
    return s;
}


bool full_of(const moe_residual_norm_config& c) { return c.post == MOE_NORM_LAYER || c.pre == MOE_NORM_LAYER; }
bool grouped_of(const moe_residual_norm_config& c) { return c.gate_rows > 0 && c.gate_rows < c.rows; }

// Backward: CTAs, and the consecutive rows of each group of warps.
RnShape backward_shape(const moe_residual_norm_config& c, int sms, int* ctas) {
    RnShape s = shape_of(c);
    s.warps = rn_warps(c.d, rn_backward_values(c.d, c.dtype, full_of(c), grouped_of(c)));
    s.groups = s.warps < 8 ? 8 / s.warps : 1;
    const int64_t most = (int64_t)sms * (s.warps * s.groups > 8 ? 1 : 2) * s.groups;
    const int64_t workers = c.rows < most ? c.rows : most;
    s.chunk = workers ? (c.rows + workers - 1) / workers : 1;
    // whole gates where a sixteenth more rows do: their gradients then need no sums over groups
    const int64_t even = grouped_of(c) ? (s.chunk + c.gate_rows - 1) / c.gate_rows * c.gate_rows : s.chunk;
    if ((even - s.chunk) * 16 <= s.chunk) s.chunk = even;
    const int64_t used = (c.rows + s.chunk - 1) / s.chunk;
    *ctas = (int)((used + s.groups - 1) / s.groups);
    return s;
}
size_t part_bytes(const moe_residual_norm_config& c, int ctas) { return (size_t)ctas * (full_of(c) ? 4 : 2) * c.d * 4; }
size_t gpart_bytes(const moe_residual_norm_config& c, int workers) { return grouped_of(c) ? (size_t)workers * 2 * c.d * 4 : 0; }  // and gsum's

// f(T()) for the config's type.
template <typename F>
cudaError_t dispatch(int dtype, F f) {
    return dtype == MOE_DTYPE_F32 ? f(float()) : dtype == MOE_DTYPE_BF16 ? f(__nv_bfloat16()) : f(__half());
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

MOE_API int moe_residual_norm_forward(const moe_residual_norm_config* c, const void* x, const void* u, const void* post_w,
                                      const void* post_b, const void* gate, const void* pre_w, const void* pre_b, void* h,
                                      void* z, float* post_stats, float* pre_stats, void* stream) {
    clear_error();
    int rc = check(c);
    if (rc) return rc;
    if ((rc = check_weights(*c, post_w, post_b, gate, pre_w, pre_b))) return rc;
    if (c->rows == 0) return MOE_OK;
    if (!x || (!h && !z)) return fail(MOE_ERR_ARG, "x is NULL, or both outputs are");
    if (!u && (c->post || c->gate_rows)) return fail(MOE_ERR_ARG, "a post norm or a gate without u");
    if ((z != nullptr) != (c->pre != MOE_NORM_NONE)) return fail(MOE_ERR_ARG, "z goes with a pre norm");
    const size_t e = dtype_size(c->dtype), bytes = (size_t)c->rows * c->d * e;
    if (!aligned(x, e) || !aligned(u, e) || !aligned(h, e) || !aligned(z, e) || !aligned(post_stats, 8) || !aligned(pre_stats, 8))
        return fail(MOE_ERR_ARG, "a pointer is not aligned (the statistics to 8 bytes, the others to their type)");
    if (!apart_or_same(h, x, bytes) || !apart_or_same(h, u, bytes) || !apart_or_same(z, x, bytes) || !apart_or_same(z, u, bytes))
        return fail(MOE_ERR_ARG, "an output shares memory with part of an input");
    const size_t vec_bytes = dtype_size(c->wdtype) * c->d, stat_bytes = 8 * (size_t)c->rows;
    const Span ps{c->post ? post_stats : nullptr, stat_bytes}, qs{c->pre ? pre_stats : nullptr, stat_bytes};
    if ((rc = check_apart({{h, bytes}, {z, bytes}, ps, qs}, {{post_w, vec_bytes}, {post_b, vec_bytes}, {gate, gate_bytes(*c)},
                                                           {pre_w, vec_bytes}, {pre_b, vec_bytes}})))
        return rc;
    if ((rc = check_apart({ps, qs}, {{x, bytes}, {u, bytes}}))) return rc;
    DeviceInfo di;
    if ((rc = check_device(&di))) return rc;
    const int vec = vector_width(*c, x, u, h, z);
    const RnForward f{x, u, h, z, reinterpret_cast<float2*>(post_stats), reinterpret_cast<float2*>(pre_stats)};
    const cudaError_t err = dispatch(c->dtype, [&](auto type) {
        return launch_residual_forward<decltype(type)>(shape_of(*c), weights_of(*c, post_w, post_b, gate, pre_w, pre_b), f, vec,
                                                       di.sms, static_cast<cudaStream_t>(stream));
    });
    return err == cudaSuccess ? MOE_OK : cuda_fail(err, "residual norm launch");
}

MOE_API int moe_residual_norm_workspace_size(const moe_residual_norm_config* c, size_t* bytes) {
    clear_error();
    const int rc = check(c);
    if (rc) return rc;
    if (!bytes) return fail(MOE_ERR_ARG, "bytes is NULL");
    int ctas;
    const RnShape s = backward_shape(*c, RN_MAX_SMS, &ctas);
    const size_t need = part_bytes(*c, ctas) + 2 * gpart_bytes(*c, ctas * s.groups), most = need > 16 ? need : 16;
    *bytes = most;
    return MOE_OK;
}

MOE_API int moe_residual_norm_backward(const moe_residual_norm_config* c, const void* dz, const void* dh, const void* u,
                                       const void* h, const void* post_w, const void* post_b, const void* gate,
                                       const void* pre_w, const float* post_stats, const float* pre_stats, void* dx,
                                       void* du, void* dpost_w, void* dpost_b, void* dgate, void* dpre_w, void* dpre_b,
                                       void* ws, size_t ws_bytes, void* stream) {
    clear_error();
    int rc = check(c);
    if (rc) return rc;
    if ((rc = check_weights(*c, post_w, post_b, gate, pre_w, nullptr))) return rc;
    const size_t e = dtype_size(c->dtype), we = dtype_size(c->wdtype), bytes = (size_t)c->rows * c->d * e;
    void* const grads[5] = {dpost_w, dpost_b, dgate, dpre_w, dpre_b};
    const bool there[5] = {c->post != 0, c->post == MOE_NORM_LAYER, c->gate_rows > 0, c->pre != 0, c->pre == MOE_NORM_LAYER};
    bool any = false;
    for (int i = 0; i < 5; ++i) {
        if (grads[i] && !there[i]) return fail(MOE_ERR_ARG, "the gradient of a weight, bias or gate that the config lacks");
        if (!aligned(grads[i], we)) return fail(MOE_ERR_ARG, "a weight's gradient is not aligned to its type");
        any |= grads[i] != nullptr;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    DeviceInfo di;
    if (c->rows == 0) {
        if (!any) return MOE_OK;
        if ((rc = check_device(&di))) return rc;
        for (int i = 0; i < 5; ++i) {
            const cudaError_t err = grads[i] && i != 2 ? cudaMemsetAsync(grads[i], 0, we * c->d, st) : cudaSuccess;
            if (err != cudaSuccess) return cuda_fail(err, "clearing the weights' gradients");
        }
        return MOE_OK;
    }
    const bool uses_u = c->post || c->gate_rows;
    if (!dx) return fail(MOE_ERR_ARG, "dx is NULL");
    if (c->pre ? !dz || !h || !pre_stats : !!dz) return fail(MOE_ERR_ARG, "dz, h and pre_stats go with a pre norm");
    if (!c->pre && !dh) return fail(MOE_ERR_ARG, "neither dz nor dh");
    if ((uses_u && !u) || (c->post && !post_stats)) return fail(MOE_ERR_ARG, "u or post_stats is NULL");
    if (!aligned(dz, e) || !aligned(dh, e) || !aligned(u, e) || !aligned(h, e) || !aligned(dx, e) || !aligned(du, e) ||
        !aligned(post_stats, 8) || !aligned(pre_stats, 8))
        return fail(MOE_ERR_ARG, "a pointer is not aligned (the statistics to 8 bytes, the others to their type)");
    for (const void* in : {dz, dh, u, h})
        if (!apart_or_same(dx, in, bytes) || !apart_or_same(du, in, bytes))
            return fail(MOE_ERR_ARG, "dx or du shares memory with part of an input");
    const size_t vec_bytes = we * c->d, stat_bytes = 8 * (size_t)c->rows;
    const Span dw[5] = {{dpost_w, vec_bytes}, {dpost_b, vec_bytes}, {dgate, gate_bytes(*c)}, {dpre_w, vec_bytes}, {dpre_b, vec_bytes}};
    const Span post_wt{post_w, vec_bytes}, post_bt{post_b, vec_bytes}, gt{gate, gate_bytes(*c)}, pre_wt{pre_w, vec_bytes};
    const Span ps{c->post ? post_stats : nullptr, stat_bytes}, qs{c->pre ? pre_stats : nullptr, stat_bytes};
    if ((rc = check_apart({{dx, bytes}, {du, bytes}, dw[0], dw[1], dw[2], dw[3], dw[4]}, {post_wt, post_bt, gt, pre_wt, ps, qs}))) return rc;
    const Span rows_in[4] = {{dz, bytes}, {dh, bytes}, {uses_u ? u : nullptr, bytes}, {c->pre ? h : nullptr, bytes}};
    if ((rc = check_apart({dw[0], dw[1], dw[2], dw[3], dw[4]}, {rows_in[0], rows_in[1], rows_in[2], rows_in[3]}))) return rc;
    if ((rc = check_device(&di))) return rc;
    const int vec = vector_width(*c, dz, dh, uses_u ? u : nullptr, c->pre ? h : nullptr, dx, du);
    int ctas;
    const RnShape s = backward_shape(*c, di.sms, &ctas);
    const bool full = full_of(*c), grouped = grouped_of(*c);
    float *part = nullptr, *gpart = nullptr, *gsum = nullptr;
    if (any) {
        const size_t p = part_bytes(*c, ctas), gp = gpart_bytes(*c, ctas * s.groups), need = p + 2 * gp;
        if (!ws) return fail(MOE_ERR_ARG, "workspace is NULL");
        if (!aligned(ws, 16)) return fail(MOE_ERR_ARG, "workspace must be 16-byte aligned");
        if (ws_bytes < need) return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
        if ((rc = check_apart({{ws, need}}, {{dx, bytes}, {du, bytes}, dw[0], dw[1], dw[2], dw[3], dw[4], post_wt, post_bt, gt, pre_wt, ps, qs,
                                             rows_in[0], rows_in[1], rows_in[2], rows_in[3]})))
            return rc;
        part = static_cast<float*>(ws);
        gpart = part + p / 4;
        gsum = gpart + gp / 4;
    }
    const RnWeights w = weights_of(*c, post_w, post_b, gate, pre_w, nullptr);
    const RnBackward b{c->pre ? dz : nullptr, dh, uses_u ? u : nullptr, c->pre ? h : nullptr,
                       reinterpret_cast<const float2*>(post_stats), reinterpret_cast<const float2*>(pre_stats), dx, du, part,
                       gpart, gsum, dgate};
    const cudaError_t err = dispatch(c->dtype, [&](auto type) {
        typedef decltype(type) T;
        const cudaError_t e0 = launch_residual_backward<T>(s, w, b, vec, full, grouped, ctas, st);
        if (e0 != cudaSuccess || !any) return e0;
        RnReduce a{part, gpart, ctas, c->d, full, grouped, w.f32, post_w, post_b, gate, dpost_w, dpost_b, dgate, dpre_w, dpre_b,
                   c->rows, c->gate_rows, s.chunk, 0, false, 1};
        if (grouped && dgate && s.chunk % c->gate_rows) {
            const int64_t places = (c->rows - 1) / s.chunk, gates = (c->rows + c->gate_rows - 1) / c->gate_rows;
            a.at_places = places < gates;
            a.shared = a.at_places ? places : gates;
        }
        while (a.each < RN_RED_ROWS && a.each * 4 < c->gate_rows / s.chunk + 2) a.each *= 2;
        const int64_t more = (a.shared * a.each + RN_RED_ROWS - 1) / RN_RED_ROWS;
        return launch_k(rn_reduce_kernel<T>, dim3((c->d + RN_RED_COLS - 1) / RN_RED_COLS, (unsigned)(2 + (more < 32 ? more : 32))),
                        dim3(RN_RED_COLS * RN_RED_ROWS), 0, st, true, a);
    });
    return err == cudaSuccess ? MOE_OK : cuda_fail(err, "residual norm backward launch");
}

}  // extern "C"
