// Global norm of a list of gradients, the factor that clips it, and clipping in place.
//
//   norm = sqrt(sum over all tensors of g^2), scale = min(1, max_norm / (norm + eps)); g = g * scale
//
// Every value is read once for the norm, read and written once for clipping: HBM traffic bounds both. A CTA takes
// chunks of 32 KB; a thread squares the 128 bytes of a chunk that it loads in fp32, adds them in chains of eight (off by 11 *
// 2^-24 of their sum at most) and that sum to a pair of floats (sum and what its rounding cut off, by the two-sum of
// Knuth and Moller), so the length of the list costs no precision. The CTAs' sums are added
// up in 64 bits by the CTA that finishes last, in the order of the CTAs: the result repeats bit for bit.
// Squares that leave fp32's range are taken again in 64 bits, so a norm that fp32 can hold is found whatever the
// values' size. 24 tensors, 149 million bf16 values: norm 47 us, 6.3 TB/s (92 % of a copy's rate); 64 bytes a thread in
// flight: 52 us. 67 tensors, 1 million values: 6.5 us, one launch and the call on the host. Clipping the long list
// after its norm: 139 us for both; 48 where the factor is 1, which ends the clipping launch at once.
#include <math.h>

#include "row_values.cuh"

namespace moe {
namespace {

constexpr int GN_THREADS = 256;
constexpr int GN_VECS = 8;                         // 16-byte pieces of a thread in flight
constexpr int GN_CHUNK = GN_THREADS * GN_VECS;     // pieces of a chunk
constexpr int GN_CTAS = 4;                         // on a SM
constexpr int GN_MOST = 2048;                      // CTAs of a launch
// Workspace: ticket (zero between calls), sum of the launches before, the CTAs' sums.
struct GnSpace {
    uint32_t ticket, pad;
    double total;
    double part[GN_MOST];
};
static_assert(sizeof(GnSpace) <= MOE_GRAD_NORM_WORKSPACE_BYTES, "workspace");

struct GnTensor {
    void* g;
    int64_t n;
};
template <int MAXT>
struct GnList {
    GnTensor t[MAXT];
    int32_t first[MAXT + 1];  // first chunk of each tensor
    uint8_t dtype[MAXT];
    int32_t count;
};
template <int MAXT>
__device__ __forceinline__ int tensor_of(const GnList<MAXT>& l, int c) {
    int lo = 0, hi = l.count - 1;  // the last tensor whose first chunk is at or before c
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (l.first[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Lists of more than GN_FIT chunks (64 MB) do not stay in L2 from the norm's pass to the clipping pass: they go through it
// as what may be replaced first. (Norm and clipping of 149 million bf16 values, 894 MB in all: 139 us; 145 without this,
// and 145 with this and chunks in ascending order in both passes; marking the list's last 16 to 96 MB as to be kept: 139
// to 146.)
constexpr int GN_FIT = 2048;
__device__ __forceinline__ uint64_t l2_policy(int chunks) {
    uint64_t first, normal;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first));
    asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(normal));
    return chunks <= GN_FIT ? normal : first;
}
template <typename P>
__device__ __forceinline__ P load_piece(const P* p, uint64_t policy) {
    static_assert(sizeof(P) == 16, "a piece");
    uint4 v;
    asm volatile("ld.global.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p), "l"(policy));
    return *reinterpret_cast<const P*>(&v);
}
template <typename P>
__device__ __forceinline__ void store_piece(P* p, const P& value, uint64_t policy) {
    const uint4 v = *reinterpret_cast<const uint4*>(&value);
    asm volatile("st.global.L2::cache_hint.v4.u32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w),
                 "l"(policy)
                 : "memory");
}

// A tensor at any address: `head` values before the first 16-byte boundary, `pieces` of 16 bytes, `tail` values.
struct GnSpan {
    int64_t head, pieces, tail;
};
__host__ __device__ __forceinline__ GnSpan span_of(const void* g, int64_t n, int size) {
    const int64_t off = (16 - (int64_t)(reinterpret_cast<uintptr_t>(g) & 15)) % 16 / size;
    GnSpan s;
    s.head = off < n ? off : n;
    s.pieces = (n - s.head) * size / 16;
    s.tail = n - s.head - s.pieces * (16 / size);
    return s;
}

// Sum of the squares of a thread's n pieces at p, a chunk's width apart, in 64 bits. A call, and the values are read again:
// inlined, on registers, it made the loop over the chunks spill.
template <typename T>
__device__ __noinline__ double wide_squares(const Pack<T, 16 / sizeof(T)>* p, int n) {
    double a = 0.0;
    for (int k = 0; k < n; ++k) {
        const Pack<T, 16 / sizeof(T)> e = p[k * GN_THREADS];
#pragma unroll
        for (int i = 0; i < 16 / (int)sizeof(T); ++i) {
            const double v = num(e.v[i]);
            a += v * v;
        }
    }
    return a;
}
// Sum of the squares of a thread's part of a chunk: in fp32 when every square that matters is a normal fp32
// number, else in 64 bits. Below 2^-110 what subnormal squares lose (2^-150 each) could matter.
template <typename T, int N, typename Sum>
__device__ __forceinline__ void add_squares(const Pack<T, 16 / sizeof(T)> (&p)[N], const Pack<T, 16 / sizeof(T)>* from, int n, Sum&& sum) {
    constexpr int VEC = 16 / sizeof(T);
    f2 acc[VEC / 2];  // one for each pair of a piece: chains of N additions, whatever the type
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) acc[i] = both<f2>(0.f);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        f2 f[VEC / 2];
        widen(p[k], f);
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) acc[i] = fma_(f[i], f[i], acc[i]);
    }
    f2 sums = add_(acc[0], acc[1]);
    if constexpr (VEC == 8) sums = add_(sums, add_(acc[2], acc[3]));
    const float s = total(sums);
    if (s >= 0x1p-110f && s <= 0x1p100f) {
        sum.add(s);
        return;
    }
    uint32_t any = 0;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) any |= reinterpret_cast<const uint32_t*>(&p[k])[i];
    if (!(any & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu))) return;  // nothing but zeros
    sum.far += wide_squares<T>(from, n);
}

// A thread's sum: hi + lo, and what fp32 cannot hold.
struct GnSum {
    float hi = 0.f, lo = 0.f;
    double far = 0.0;
    __device__ __forceinline__ void add(float s) {
        const float t = __fadd_rn(hi, s), b = __fsub_rn(t, hi);
        lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(s, b));  // what the sum's rounding cut off
        hi = t;
    }
    __device__ __forceinline__ double value() const { return (double)hi + lo + far; }
};

template <typename T>
__device__ __forceinline__ void chunk_squares(const GnTensor& t, int64_t chunk, uint64_t policy, GnSum& sum) {
    constexpr int VEC = 16 / sizeof(T);
    const GnSpan sp = span_of(t.g, t.n, sizeof(T));
    const T* const g = static_cast<const T*>(t.g);
    const Pack<T, VEC>* const body = reinterpret_cast<const Pack<T, VEC>*>(g + sp.head);
    const int64_t at = chunk * GN_CHUNK;
    Pack<T, VEC> p[GN_VECS];
    if (at + GN_CHUNK <= sp.pieces) {
#pragma unroll
        for (int k = 0; k < GN_VECS; ++k) p[k] = load_piece(body + (at + k * GN_THREADS + threadIdx.x), policy);
    } else {
#pragma unroll
        for (int k = 0; k < GN_VECS; ++k) {
            const int64_t i = at + k * GN_THREADS + threadIdx.x;
            if (i < sp.pieces) p[k] = load_piece(body + i, policy);
            else memset(&p[k], 0, sizeof(p[k]));
        }
    }
    const int64_t left = sp.pieces - at - threadIdx.x;
    add_squares<T>(p, body + at + threadIdx.x, left <= 0 ? 0 : left >= GN_CHUNK ? GN_VECS : min(GN_VECS, (int)((left + GN_THREADS - 1) / GN_THREADS)), sum);
    // the values around the pieces: fewer than 8 on each side, in the first chunk
    if (chunk == 0 && threadIdx.x < 16) {
        const int64_t i = threadIdx.x < 8 ? threadIdx.x : threadIdx.x - 8;
        const bool mine = threadIdx.x < 8 ? i < sp.head : i < sp.tail;
        const int64_t e = threadIdx.x < 8 ? i : t.n - sp.tail + i;
        if (mine) {
            const double v = num(g[e]);
            sum.far += v * v;
        }
    }
}

__device__ __forceinline__ double warp_total(double a) {
#pragma unroll
    for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    return a;
}
__device__ __forceinline__ double cta_total(double a, double* red) {  // valid in thread 0
    a = warp_total(a);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
    __syncthreads();
    a = 0.0;
    if (threadIdx.x == 0)
        for (int i = 0; i < GN_THREADS / 32; ++i) a += red[i];
    return a;
}

struct GnEnd {
    double max_norm, eps;
    int first, last;  // whether this launch is the call's first, and its last
    float* out;
};

template <int MAXT>
__global__ void __launch_bounds__(GN_THREADS, GN_CTAS)
    grad_norm_kernel(const __grid_constant__ GnList<MAXT> l, const GnEnd end, GnSpace* ws) {
    __shared__ double red[2][GN_THREADS / 32];
    __shared__ bool am_last;
    griddep_wait();
    griddep_launch();
    GnSum sum;
    const uint64_t policy = l2_policy(l.first[l.count]);
    for (int c = blockIdx.x; c < l.first[l.count]; c += gridDim.x) {
        const int i = tensor_of(l, c);
        const int64_t chunk = c - l.first[i];
        if (l.dtype[i] == MOE_DTYPE_F32) chunk_squares<float>(l.t[i], chunk, policy, sum);
        else if (l.dtype[i] == MOE_DTYPE_BF16) chunk_squares<__nv_bfloat16>(l.t[i], chunk, policy, sum);
        else chunk_squares<__half>(l.t[i], chunk, policy, sum);
    }
    const double mine = cta_total(sum.value(), red[0]);
    if (threadIdx.x == 0) {
        ws->part[blockIdx.x] = mine;
        __threadfence();
        am_last = atomicAdd(&ws->ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!am_last) return;
    __threadfence();
    double a = 0.0;
    for (int i = threadIdx.x; i < (int)gridDim.x; i += GN_THREADS) a += __ldcg(&ws->part[i]);
    a = cta_total(a, red[1]);
    if (threadIdx.x) return;
    if (!end.first) a += ws->total;
    ws->total = a;
    ws->ticket = 0;
    if (!end.last) return;
    const double norm = sqrt(a), f = end.max_norm / (norm + end.eps);
    end.out[0] = (float)norm;
    // 1 also for infinity / infinity (no limit) and 0 / 0 (nothing to scale); a norm that is NaN makes the factor so
    end.out[1] = f < 1.0 || norm != norm ? (float)f : 1.0f;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const GnTensor& t, int64_t chunk, uint64_t policy, float scale) {
    constexpr int VEC = 16 / sizeof(T);
    const GnSpan sp = span_of(t.g, t.n, sizeof(T));
    T* const g = static_cast<T*>(t.g);
    Pack<T, VEC>* const body = reinterpret_cast<Pack<T, VEC>*>(g + sp.head);
    const f2 by = pair(scale, scale);
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {  // half the pieces at a time: all of them took more registers than there are
        const int64_t at = chunk * GN_CHUNK + half * (GN_CHUNK / 2) + threadIdx.x;
        Pack<T, VEC> p[GN_VECS / 2];
#pragma unroll
        for (int k = 0; k < GN_VECS / 2; ++k)
            if (at + k * GN_THREADS < sp.pieces) p[k] = load_piece(body + (at + k * GN_THREADS), policy);
#pragma unroll
        for (int k = 0; k < GN_VECS / 2; ++k) {
            if (at + k * GN_THREADS >= sp.pieces) break;
            f2 f[VEC / 2];
            widen(p[k], f);
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) f[i] = mul_(f[i], by);
            store_piece(body + (at + k * GN_THREADS), narrow<T, VEC>(f), policy);
        }
    }
    if (chunk == 0 && threadIdx.x < 16) {
        const int64_t i = threadIdx.x < 8 ? threadIdx.x : threadIdx.x - 8;
        const bool mine = threadIdx.x < 8 ? i < sp.head : i < sp.tail;
        const int64_t e = threadIdx.x < 8 ? i : t.n - sp.tail + i;
        if (mine) put(g[e], num(g[e]) * scale);
    }
}

// Chunks from the last to the first: some of what the norm's pass read last is still in L2.
template <int MAXT>
__global__ void __launch_bounds__(GN_THREADS, GN_CTAS)
    grad_clip_kernel(const __grid_constant__ GnList<MAXT> l, const float* scale) {
    griddep_wait();
    griddep_launch();
    const float s = *scale;
    if (s == 1.0f) return;  // the usual step of a settled run: every bit stays, a NaN's too, and nothing is read or written
    const uint64_t policy = l2_policy(l.first[l.count]);
    for (int c = l.first[l.count] - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
        const int i = tensor_of(l, c);
        const int64_t chunk = c - l.first[i];
        if (l.dtype[i] == MOE_DTYPE_F32) chunk_scale<float>(l.t[i], chunk, policy, s);
        else if (l.dtype[i] == MOE_DTYPE_BF16) chunk_scale<__nv_bfloat16>(l.t[i], chunk, policy, s);
        else chunk_scale<__half>(l.t[i], chunk, policy, s);
    }
}

// A short list takes the small parameter block; longer ones take several launches.
constexpr int GN_SMALL = 72, GN_LARGE = 1300;
static_assert(sizeof(GnList<GN_LARGE>) + sizeof(GnEnd) < 32000, "launch parameters");

// `apart`: `bytes` of the caller's that lie in no tensor.
int check_list(const moe_grad_tensor* ts, int32_t count, const void* apart, size_t bytes, int64_t* values) {
    if (count < 0) return fail(MOE_ERR_ARG, "count=%d must be >= 0", count);
    if (count && !ts) return fail(MOE_ERR_ARG, "tensors is NULL");
    *values = 0;
    for (int i = 0; i < count; ++i) {
        const moe_grad_tensor& t = ts[i];
        if (t.n < 0) return fail(MOE_ERR_ARG, "tensor %d: n=%lld must be >= 0", i, (long long)t.n);
        if (t.dtype != MOE_DTYPE_F32 && t.dtype != MOE_DTYPE_BF16 && t.dtype != MOE_DTYPE_F16)
            return fail(MOE_ERR_ARG, "tensor %d: dtype=%d is not a MOE_DTYPE", i, t.dtype);
        if (t.reserved) return fail(MOE_ERR_ARG, "reserved fields must be zero");
        if (t.n == 0) continue;
        if (!t.g) return fail(MOE_ERR_ARG, "tensor %d: g is NULL", i);
        if (!aligned(t.g, dtype_size(t.dtype))) return fail(MOE_ERR_ARG, "tensor %d is not aligned to its type", i);
        const uintptr_t from = reinterpret_cast<uintptr_t>(t.g), at = reinterpret_cast<uintptr_t>(apart);
        if (apart && at + bytes > from && at < from + dtype_size(t.dtype) * (size_t)t.n)
            return fail(MOE_ERR_ARG, "tensor %d holds the factor or the norm", i);
        *values += t.n;
    }
    return MOE_OK;
}

// Calls run(list, chunks, last) for each launch's part of the list.
template <int MAXT, typename Run>
int over_list(const moe_grad_tensor* ts, int count, Run run) {
    GnList<MAXT> l;
    for (int i = 0;;) {
        int k = 0;
        int64_t chunks = 0;
        for (; i < count && k < MAXT; ++i) {
            if (ts[i].n == 0) continue;
            const int64_t pieces = span_of(ts[i].g, ts[i].n, (int)dtype_size(ts[i].dtype)).pieces;
            const int64_t more = pieces ? (pieces + GN_CHUNK - 1) / GN_CHUNK : 1;
            if (chunks + more > INT_MAX / 2) break;
            l.t[k] = GnTensor{ts[i].g, ts[i].n};
            l.dtype[k] = (uint8_t)ts[i].dtype;
            l.first[k++] = (int32_t)chunks;
            chunks += more;
        }
        if (k == 0 && i < count) return fail(MOE_ERR_ARG, "tensor %d is too long", i);
        while (i < count && ts[i].n == 0) ++i;
        l.first[k] = (int32_t)chunks;
        l.count = k;
        const int rc = run(l, (int)chunks, i >= count);
        if (rc || i >= count) return rc;
    }
}

int grid_for(const DeviceInfo& di, int chunks) {
    int most = di.sms * GN_CTAS < GN_MOST ? di.sms * GN_CTAS : GN_MOST;
    return chunks < 1 ? 1 : chunks < most ? chunks : most;
}

template <int MAXT>
int norm_list(const moe_grad_norm_config& c, const moe_grad_tensor* ts, int count, float* out, void* ws,
              const DeviceInfo& di, cudaStream_t st) {
    bool first = true;
    return over_list<MAXT>(ts, count, [&](const GnList<MAXT>& l, int chunks, bool last) {
        const GnEnd end{c.max_norm, c.eps, first, last, out};
        first = false;
        const cudaError_t e = launch_k(grad_norm_kernel<MAXT>, dim3(grid_for(di, chunks)), dim3(GN_THREADS), 0, st, true,
                                       l, end, static_cast<GnSpace*>(ws));
        return e == cudaSuccess ? MOE_OK : cuda_fail(e, "gradient norm launch");
    });
}

template <int MAXT>
int clip_list(const moe_grad_tensor* ts, int count, const float* scale, const DeviceInfo& di, cudaStream_t st) {
    return over_list<MAXT>(ts, count, [&](const GnList<MAXT>& l, int chunks, bool) {
        const cudaError_t e =
            launch_k(grad_clip_kernel<MAXT>, dim3(grid_for(di, chunks)), dim3(GN_THREADS), 0, st, true, l, scale);
        return e == cudaSuccess ? MOE_OK : cuda_fail(e, "gradient clipping launch");
    });
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

MOE_API int moe_grad_norm(const moe_grad_norm_config* c, const moe_grad_tensor* ts, int32_t count, float* out, void* ws,
                          size_t ws_bytes, void* stream) {
    clear_error();
    if (!c) return fail(MOE_ERR_ARG, "config is NULL");
    if (!(c->max_norm >= 0)) return fail(MOE_ERR_ARG, "max_norm=%g must be >= 0", c->max_norm);
    if (!(c->eps >= 0) || !isfinite(c->eps)) return fail(MOE_ERR_ARG, "eps=%g must be >= 0 and finite", c->eps);
    for (int i = 0; i < 4; ++i)
        if (c->reserved[i]) return fail(MOE_ERR_ARG, "reserved fields must be zero");
    int64_t values;
    int rc = check_list(ts, count, out, 8, &values);
    if (rc) return rc;
    if (!out || !ws) return fail(MOE_ERR_ARG, "out or workspace is NULL");
    if (!aligned(out, 4) || !aligned(ws, 16)) return fail(MOE_ERR_ARG, "out must be 4-byte and ws 16-byte aligned");
    if (ws_bytes < MOE_GRAD_NORM_WORKSPACE_BYTES)
        return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %d", ws_bytes, MOE_GRAD_NORM_WORKSPACE_BYTES);
    DeviceInfo di;
    if ((rc = check_device(&di))) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return count <= GN_SMALL ? norm_list<GN_SMALL>(*c, ts, count, out, ws, di, st)
                             : norm_list<GN_LARGE>(*c, ts, count, out, ws, di, st);
}

MOE_API int moe_grad_clip(const moe_grad_tensor* ts, int32_t count, const float* scale, void* stream) {
    clear_error();
    int64_t values;
    int rc = check_list(ts, count, scale, 4, &values);
    if (rc) return rc;
    if (!scale) return fail(MOE_ERR_ARG, "scale is NULL");
    if (!aligned(scale, 4)) return fail(MOE_ERR_ARG, "scale must be 4-byte aligned");
    if (values == 0) return MOE_OK;
    DeviceInfo di;
    if ((rc = check_device(&di))) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return count <= GN_SMALL ? clip_list<GN_SMALL>(ts, count, scale, di, st)
                             : clip_list<GN_LARGE>(ts, count, scale, di, st);
}

}  // extern "C"
