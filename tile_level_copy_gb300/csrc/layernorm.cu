// Layer norm over rows, forward and backward, with the reduction of the weight's and bias's gradients.
//
//   forward   mean = sum x / d, rstd = 1 / sqrt(sum (x - mean)^2 / d + eps), y = (x - mean) rstd w + b
//   backward  xh = (x - mean) rstd, gy = dy w
//             dx = rstd (gy - sum(gy) / d - xh sum(gy xh) / d), dw = sum_rows dy xh, db = sum_rows dy
//
// The forward pass reads x and writes y, the backward pass reads x and dy and writes dx: both are
// bound by HBM. A group of threads holds its whole row in registers (16 values a thread, 32 for rows above 8192), so the
// variance is the mean of squared differences (no cancellation) without a second read, and the
// next row's values are loaded while this row's sums are taken. Groups keep their columns'
// weights, and in the backward pass their columns' partial sums of dw and db, in registers over all
// their rows; the partial sums of each CTA are added up in a second launch in CTA order.
#include "host_internal.h"
#include "moe_internal.cuh"

#include <cuda_fp16.h>

namespace moe {
namespace {

constexpr int LN_MAX_THREADS = 512;
constexpr int LN_WIDE = 16 * LN_MAX_THREADS;  // rows above this take 32 values a thread
constexpr int LN_MAX_D = 32 * LN_MAX_THREADS;
constexpr int LN_THREADS = 256;   // threads of a CTA when a row takes fewer
constexpr int LN_RED_COLS = 32;   // columns of a CTA of the second launch
constexpr int LN_RED_ROWS = 16;   // partial sums it adds side by side

__device__ __forceinline__ float num(float v) { return v; }
__device__ __forceinline__ float num(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float num(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half rounded<__half>(float v) { return __float2half_rn(v); }

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
};

// How the threads of a launch share the rows: `tpr` threads a row (a power of two up to 32, or whole
// warps), `groups` rows at a time in a CTA.
struct LnShape {
    int64_t rows;
    int d, tpr, groups;
    float eps, inv_d;
};

// A thread's E values of a row as VEC-wide pieces: piece q covers columns (q * tpr + t) * VEC...
template <typename T, int VEC, int E>
struct RowPart {
    static constexpr int NP = E / VEC;
    Pack<T, VEC> p[NP];
    __device__ __forceinline__ void load(const T* row, int t, const LnShape& s) {
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            const int c = (q * s.tpr + t) * VEC;
            if (c < s.d) p[q] = *reinterpret_cast<const Pack<T, VEC>*>(row + c);
        }
    }
    __device__ __forceinline__ void floats(float (&f)[E], int t, const LnShape& s) const {
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            const bool in = (q * s.tpr + t) * VEC < s.d;
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[q * VEC + j] = in ? num(p[q].v[j]) : 0.f;
        }
    }
};

template <typename T, int VEC, int E>
__device__ __forceinline__ void store_row(T* row, const float (&f)[E], int t, const LnShape& s) {
#pragma unroll
    for (int q = 0; q < E / VEC; ++q) {
        const int c = (q * s.tpr + t) * VEC;
        if (c >= s.d) continue;
        Pack<T, VEC> o;
#pragma unroll
        for (int j = 0; j < VEC; ++j) o.v[j] = rounded<T>(f[q * VEC + j]);
        *reinterpret_cast<Pack<T, VEC>*>(row + c) = o;
    }
}

// Weights of a thread's columns (w null: `none`).
template <typename T, int VEC, int E>
__device__ __forceinline__ void load_weights(const void* w, bool f32, float none, float (&f)[E], int t,
                                             const LnShape& s) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int c = ((i / VEC) * s.tpr + t) * VEC + i % VEC;
        f[i] = none;
        if (w && c < s.d) f[i] = f32 ? static_cast<const float*>(w)[c] : num(static_cast<const T*>(w)[c]);
    }
}

// Sum of a and b over a row's group of threads, the same in all of them. Groups of whole warps pass
// their warps' sums through `red` (32 float2 a group, used alternately by `flip` so that one
// barrier a sum is enough).
__device__ __forceinline__ float2 group_sum(float a, float b, int tpr, int group, float2* red, int& flip) {
    for (int o = min(tpr, 32) >> 1; o; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (tpr <= 32) return make_float2(a, b);
    const int warps = tpr >> 5, w = (threadIdx.x % tpr) >> 5, lane = threadIdx.x & 31;
    float2* r = red + (flip * (blockDim.x / 32)) + group * warps;
    flip ^= 1;
    if (lane == 0) r[w] = make_float2(a, b);
    named_bar_sync(1 + group, tpr);
    float2 v = lane < warps ? r[lane] : make_float2(0.f, 0.f);
    for (int o = 16; o; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    return v;
}

template <typename T, int VEC, int E>
__global__ void __launch_bounds__(LN_MAX_THREADS) ln_forward_kernel(LnShape s, const T* x, const void* w, const void* b,
                                                          bool wf32, T* y, float* mean, float* rstd) {
    __shared__ float2 red[64];
    griddep_wait();
    griddep_launch();
    const int t = threadIdx.x % s.tpr, group = threadIdx.x / s.tpr;
    const int64_t stride = (int64_t)gridDim.x * s.groups;
    float wf[E], bf[E];
    load_weights<T, VEC, E>(w, wf32, 1.f, wf, t, s);
    load_weights<T, VEC, E>(b, wf32, 0.f, bf, t, s);
    int flip = 0;
    RowPart<T, VEC, E> next;
    int64_t r = (int64_t)blockIdx.x * s.groups + group;
    // groups that share a warp take part in its shuffles until all of them are done
    const int64_t last = s.tpr < 32 ? r - group % (32 / s.tpr) : r;
    if (r < s.rows) next.load(x + r * s.d, t, s);
    for (int64_t r0 = last; r0 < s.rows; r0 += stride, r += stride) {
        const RowPart<T, VEC, E> part = next;
        const bool in = r < s.rows;
        if (r + stride < s.rows) next.load(x + (r + stride) * s.d, t, s);
        float f[E];
        part.floats(f, t, s);
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) a += f[i];
        const float mu = group_sum(a, 0.f, s.tpr, group, red, flip).x * s.inv_d;
        a = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = ((i / VEC) * s.tpr + t) * VEC;
            f[i] = c < s.d ? f[i] - mu : 0.f;
            a = fmaf(f[i], f[i], a);
        }
        const float var = group_sum(a, 0.f, s.tpr, group, red, flip).x * s.inv_d;
        const float rs = 1.0f / sqrtf(var + s.eps);
        if (!in) continue;
#pragma unroll
        for (int i = 0; i < E; ++i) f[i] = fmaf(f[i] * rs, wf[i], bf[i]);
        store_row<T, VEC>(y + r * s.d, f, t, s);
        if (t == 0) {
            if (mean) mean[r] = mu;
            if (rstd) rstd[r] = rs;
        }
    }
}

template <typename T, int VEC, int E>
__global__ void __launch_bounds__(LN_MAX_THREADS) ln_backward_kernel(LnShape s, const T* dy, const T* x, const void* w, bool wf32,
                                                           const float* mean, const float* rstd, T* dx, float* part) {
    __shared__ float2 red[64];
    griddep_wait();
    griddep_launch();
    const int t = threadIdx.x % s.tpr, group = threadIdx.x / s.tpr;
    const int64_t stride = (int64_t)gridDim.x * s.groups;
    float wf[E], dw[E], db[E];
    load_weights<T, VEC, E>(w, wf32, 1.f, wf, t, s);
#pragma unroll
    for (int i = 0; i < E; ++i) dw[i] = db[i] = 0.f;
    int flip = 0;
    RowPart<T, VEC, E> nx, ny;
    float nmu = 0.f, nrs = 0.f;
    int64_t r = (int64_t)blockIdx.x * s.groups + group;
    const int64_t last = s.tpr < 32 ? r - group % (32 / s.tpr) : r;
    auto fetch = [&](int64_t q) {
        nx.load(x + q * s.d, t, s);
        ny.load(dy + q * s.d, t, s);
        nmu = mean[q];
        nrs = rstd[q];
    };
    if (r < s.rows) fetch(r);
    for (int64_t r0 = last; r0 < s.rows; r0 += stride, r += stride) {
        const RowPart<T, VEC, E> px = nx, py = ny;
        const float mu = nmu, rs = nrs;
        const bool in = r < s.rows;
        if (r + stride < s.rows) fetch(r + stride);
        float xh[E], g[E];
        px.floats(xh, t, s);
        py.floats(g, t, s);
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = ((i / VEC) * s.tpr + t) * VEC;
            const bool on = in && c < s.d;
            xh[i] = on ? (xh[i] - mu) * rs : 0.f;
            g[i] = on ? g[i] : 0.f;
            dw[i] = fmaf(g[i], xh[i], dw[i]);
            db[i] += g[i];
            g[i] *= wf[i];
            a += g[i];
            b = fmaf(g[i], xh[i], b);
        }
        const float2 c = group_sum(a, b, s.tpr, group, red, flip);
        if (!in) continue;
        const float c1 = c.x * s.inv_d, c2 = c.y * s.inv_d;
#pragma unroll
        for (int i = 0; i < E; ++i) g[i] = rs * (g[i] - c1 - xh[i] * c2);
        store_row<T, VEC>(dx + r * s.d, g, t, s);
    }
    if (!part) return;
    // this CTA's sums: its groups' one after another, so that the order is the same every time
    float* pw = part + (size_t)blockIdx.x * 2 * s.d;
    for (int q = 0; q < s.groups; ++q) {
        if (group == q) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int c = ((i / VEC) * s.tpr + t) * VEC + i % VEC;
                if (c >= s.d) continue;
                pw[c] = q ? pw[c] + dw[i] : dw[i];
                pw[s.d + c] = q ? pw[s.d + c] + db[i] : db[i];
            }
        }
        __syncthreads();
    }
}

// dw and db from the CTAs' partial sums [parts][2][d]: CTA (column block, 0 for dw / 1 for db).
template <typename T>
__global__ void __launch_bounds__(LN_RED_COLS* LN_RED_ROWS)
    ln_reduce_kernel(const float* part, int parts, int d, bool wf32, void* dw, void* db) {
    __shared__ float acc[LN_RED_ROWS][LN_RED_COLS];
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x % LN_RED_COLS, row = threadIdx.x / LN_RED_COLS;
    const int c = blockIdx.x * LN_RED_COLS + lane;
    void* out = blockIdx.y ? db : dw;
    float a = 0.f;
    if (c < d)
        for (int q = row; q < parts; q += LN_RED_ROWS) a += part[((size_t)q * 2 + blockIdx.y) * d + c];
    acc[row][lane] = a;
    __syncthreads();
    if (row || c >= d || !out) return;
    a = 0.f;
    for (int q = 0; q < LN_RED_ROWS; ++q) a += acc[q][lane];
    if (wf32) static_cast<float*>(out)[c] = a;
    else static_cast<T*>(out)[c] = rounded<T>(a);
}

size_t dtype_size(int t) { return t == MOE_DTYPE_F32 ? 4 : 2; }

int check(const moe_layernorm_config* c) {
    if (!c) return fail(MOE_ERR_ARG, "config is NULL");
    if (c->rows < 0) return fail(MOE_ERR_ARG, "rows=%lld must be >= 0", (long long)c->rows);
    if (c->d < 1 || c->d > LN_MAX_D) return fail(MOE_ERR_ARG, "d=%d must be in [1, %d]", c->d, LN_MAX_D);
    if (c->dtype != MOE_DTYPE_F32 && c->dtype != MOE_DTYPE_BF16 && c->dtype != MOE_DTYPE_F16)
        return fail(MOE_ERR_ARG, "dtype=%d is not a MOE_DTYPE", c->dtype);
    if (c->wdtype != MOE_DTYPE_F32 && c->wdtype != c->dtype)
        return fail(MOE_ERR_ARG, "wdtype=%d must be fp32 or dtype", c->wdtype);
    if (!(c->eps >= 0)) return fail(MOE_ERR_ARG, "eps=%g must be >= 0", (double)c->eps);
    for (int i = 0; i < 4; ++i)
        if (c->reserved[i]) return fail(MOE_ERR_ARG, "reserved fields must be zero");
    return MOE_OK;
}

// Widest piece (in values) that divides the rows and keeps every row's pieces aligned.
int vector_width(const moe_layernorm_config& c, const void* a, const void* b, const void* e) {
    const size_t size = dtype_size(c.dtype);
    for (int v = (int)(16 / size); v > 1; v /= 2)
        if (c.d % v == 0 && aligned(a, v * size) && aligned(b, v * size) && aligned(e, v * size)) return v;
    return 1;
}

LnShape shape_of(const moe_layernorm_config& c, int vec, int threads) {
    LnShape s;
    s.rows = c.rows;
    s.d = c.d;
    s.eps = c.eps;
    s.inv_d = 1.0f / (float)c.d;
    // 16 or 32 values a thread, in whole pieces: np pieces of vec values each
    const int values = c.d > LN_WIDE ? 32 : 16;
    const int np = values / vec, pieces = (c.d + vec - 1) / vec;
    int tpr = (pieces + np - 1) / np;
    if (tpr <= 32) {
        int p2 = 1;
        while (p2 < tpr) p2 *= 2;
        tpr = p2;
    } else {
        tpr = (tpr + 31) / 32 * 32;
    }
    s.tpr = tpr;
    s.groups = tpr < threads ? threads / tpr : 1;
    if (tpr > 32 && s.groups > 8) s.groups = 8;
    return s;
}

int check_device(DeviceInfo* di) {
    const int rc = device_info(di);
    if (rc) return rc;
    return di->supported ? MOE_OK : fail(MOE_ERR_DEVICE, "current device is not sm_103 (GB300)");
}

// f(Pack<T, VEC>, E) for the config's type, piece width and values a thread.
template <int N>
struct Int {
    static constexpr int value = N;
};
template <typename E, typename F>
cudaError_t dispatch_type(int dtype, int vec, E n, F f) {
    if (dtype == MOE_DTYPE_F32) {
        if (vec == 4) return f(Pack<float, 4>(), n);
        if (vec == 2) return f(Pack<float, 2>(), n);
        return f(Pack<float, 1>(), n);
    }
    if (dtype == MOE_DTYPE_BF16) {
        if (vec == 8) return f(Pack<__nv_bfloat16, 8>(), n);
        if (vec == 4) return f(Pack<__nv_bfloat16, 4>(), n);
        if (vec == 2) return f(Pack<__nv_bfloat16, 2>(), n);
        return f(Pack<__nv_bfloat16, 1>(), n);
    }
    if (vec == 8) return f(Pack<__half, 8>(), n);
    if (vec == 4) return f(Pack<__half, 4>(), n);
    if (vec == 2) return f(Pack<__half, 2>(), n);
    return f(Pack<__half, 1>(), n);
}

template <typename F>
cudaError_t dispatch(const moe_layernorm_config& c, int vec, F f) {
    return c.d > LN_WIDE ? dispatch_type(c.dtype, vec, Int<32>(), f) : dispatch_type(c.dtype, vec, Int<16>(), f);
}

int64_t ctas_for(const LnShape& s, int64_t most) {
    const int64_t n = (s.rows + s.groups - 1) / s.groups;
    return n < most ? n : most;
}

// CTAs of the backward launch: as many as the device holds at once.
int backward_ctas(const LnShape& s, int sms) {
    const int threads = s.tpr * s.groups;
    return (int)ctas_for(s, (int64_t)sms * (threads > 512 ? 1 : 512 / threads < 1 ? 1 : 512 / threads));
}
constexpr int LN_MAX_SMS = 256;

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

MOE_API int moe_layernorm_forward(const moe_layernorm_config* c, const void* x, const void* w, const void* b, void* y,
                                  float* mean, float* rstd, void* stream) {
    clear_error();
    int rc = check(c);
    if (rc) return rc;
    if (c->rows == 0) return MOE_OK;
    if (!x || !y) return fail(MOE_ERR_ARG, "NULL input or output pointer");
    const size_t e = dtype_size(c->dtype), we = dtype_size(c->wdtype);
    if (!aligned(x, e) || !aligned(y, e) || !aligned(w, we) || !aligned(b, we) || !aligned(mean, 4) || !aligned(rstd, 4))
        return fail(MOE_ERR_ARG, "a pointer is not aligned to its type");
    DeviceInfo di;
    if ((rc = check_device(&di))) return rc;
    const int vec = vector_width(*c, x, y, y);
    const LnShape s = shape_of(*c, vec, LN_THREADS);
    const int threads = s.tpr * s.groups;
    const int64_t ctas = ctas_for(s, (int64_t)di.sms * (1024 / threads < 1 ? 1 : 1024 / threads));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t err = dispatch(*c, vec, [&](auto pk, auto n) {
        typedef decltype(pk) P;
        typedef std::remove_reference_t<decltype(pk.v[0])> T;
        constexpr int V = (int)(sizeof(P) / sizeof(T)), E = decltype(n)::value;
        return launch_k(ln_forward_kernel<T, V, E>, dim3((unsigned)ctas), dim3(threads), 0, st, true, s,
                        static_cast<const T*>(x), w, b, c->wdtype == MOE_DTYPE_F32, static_cast<T*>(y), mean, rstd);
    });
    return err == cudaSuccess ? MOE_OK : cuda_fail(err, "layer norm launch");
}

MOE_API int moe_layernorm_workspace_size(const moe_layernorm_config* c, size_t* bytes) {
    clear_error();
    const int rc = check(c);
    if (rc) return rc;
    if (!bytes) return fail(MOE_ERR_ARG, "bytes is NULL");
    // a backward launch's CTAs are largest for the narrowest pieces' fewest threads: 512 threads an
    // SM of at least 64, on the largest device, and never more than the rows
    const int64_t most = (int64_t)LN_MAX_SMS * 8;
    const int64_t n = c->rows < most ? c->rows : most;
    *bytes = (size_t)(n < 1 ? 1 : n) * 2 * c->d * 4;
    return MOE_OK;
}

MOE_API int moe_layernorm_backward(const moe_layernorm_config* c, const void* dy, const void* x, const void* w,
                                   const float* mean, const float* rstd, void* dx, void* dw, void* db, void* ws,
                                   size_t ws_bytes, void* stream) {
    clear_error();
    int rc = check(c);
    if (rc) return rc;
    const size_t e = dtype_size(c->dtype), we = dtype_size(c->wdtype);
    if (!aligned(dw, we) || !aligned(db, we) || !aligned(w, we))
        return fail(MOE_ERR_ARG, "a pointer is not aligned to its type");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    DeviceInfo di;
    if (c->rows == 0) {
        if (!dw && !db) return MOE_OK;
        if ((rc = check_device(&di))) return rc;
        cudaError_t err = dw ? cudaMemsetAsync(dw, 0, we * c->d, st) : cudaSuccess;
        if (err == cudaSuccess && db) err = cudaMemsetAsync(db, 0, we * c->d, st);
        return err == cudaSuccess ? MOE_OK : cuda_fail(err, "clearing the weight gradients");
    }
    if (!dy || !x || !mean || !rstd || !dx) return fail(MOE_ERR_ARG, "NULL input or output pointer");
    if (!aligned(dy, e) || !aligned(x, e) || !aligned(dx, e) || !aligned(mean, 4) || !aligned(rstd, 4))
        return fail(MOE_ERR_ARG, "a pointer is not aligned to its type");
    if ((rc = check_device(&di))) return rc;
    const int vec = vector_width(*c, dy, x, dx);
    const LnShape s = shape_of(*c, vec, LN_THREADS);
    const int ctas = backward_ctas(s, di.sms);
    float* part = nullptr;
    if (dw || db) {
        const size_t need = (size_t)ctas * 2 * c->d * 4;
        if (!ws) return fail(MOE_ERR_ARG, "workspace is NULL");
        if (!aligned(ws, 16)) return fail(MOE_ERR_ARG, "workspace must be 16-byte aligned");
        if (ws_bytes < need) return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
        part = static_cast<float*>(ws);
    }
    const bool wf32 = c->wdtype == MOE_DTYPE_F32;
    const cudaError_t err = dispatch(*c, vec, [&](auto pk, auto n) {
        typedef decltype(pk) P;
        typedef std::remove_reference_t<decltype(pk.v[0])> T;
        constexpr int V = (int)(sizeof(P) / sizeof(T)), E = decltype(n)::value;
        cudaError_t e1 = launch_k(ln_backward_kernel<T, V, E>, dim3(ctas), dim3(s.tpr * s.groups), 0, st, true, s,
                                  static_cast<const T*>(dy), static_cast<const T*>(x), w, wf32, mean, rstd,
                                  static_cast<T*>(dx), part);
        if (e1 != cudaSuccess || !part) return e1;
        return launch_k(ln_reduce_kernel<T>, dim3((c->d + LN_RED_COLS - 1) / LN_RED_COLS, 2),
                        dim3(LN_RED_COLS * LN_RED_ROWS), 0, st, true, (const float*)part, ctas, c->d, wf32, dw, db);
    });
    return err == cudaSuccess ? MOE_OK : cuda_fail(err, "layer norm backward launch");
}

}  // extern "C"
