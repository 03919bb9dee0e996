// Layer norm over rows, forward and backward, with the reduction of the weight's and bias's gradients.
//
//   forward   mean = sum x / d, rstd = 1 / sqrt(sum (x - mean)^2 / d + eps), y = (x - mean) rstd w + b
//   backward  xh = (x - mean) rstd, gy = dy w
//             dx = rstd (gy - sum(gy) / d - xh sum(gy xh) / d), dw = sum_rows dy xh, db = sum_rows dy
//
// The forward pass reads x and writes y, the backward pass reads x and dy and writes dx: HBM would bound both if
// enough loads were in flight all the time. They wait instead; see the figures below. Sums and products go two at a
// time (f32x2).
//
// Forward: a row lies in the registers of as many warps as hold it with 32 values a thread, so the
// variance is the mean of squared differences without a second read, and all of a row's loads are in
// flight at once. Weights come from L1. 16384 x 4096 bf16 take 59 us, 4.5 TB/s, where the memory needs 40 us and
// the instructions (21 a value) fill 64 % of the issue slots. What is left are waits: a warp loads its row, waits for
// it (3.4 of the 11.3 cycles between two instructions), reduces twice and stores, with no load of its next row
// under way.
// Backward: a thread keeps the same columns over all its rows, with their partial sums of dw and db
// in registers, and takes several rows at a time (32 values in all) so that one reduction and one
// barrier serve all of them; the rows come through shared memory by cp.async, two batches ahead. The
// CTAs' partial sums are added up in CTA order by a second launch. 16384 x 2048 bf16 take 49 us, 4.1 TB/s, where
// the memory needs 30 us and the instructions (21 a value) fill 45 % of the issue slots: 128 registers a thread
// leave 15 warps a SM, and of the 8.4 cycles between two instructions of one it waits 2.6 for loads and
// 1.2 at the barrier that a batch of rows has. The second launch is 7 us of it under the profiler. Above 4096 columns
// the 16-bit kernels spill: as many values take 73 us in rows of 8192 and 117 us in rows of 16384.
#include "row_values.cuh"

namespace moe {
namespace {

constexpr int LN_FWD_THREADS = 256;
constexpr int LN_BWD_THREADS = 256;  // a row above 2048 values takes up to 512
constexpr int LN_BWD_MOST = 512;
constexpr int LN_MAX_D = 16384;
constexpr int LN_RED_COLS = 32;   // columns of a CTA of the reduction
constexpr int LN_RED_ROWS = 32;   // partial sums it adds side by side

// How a launch's threads share the rows: groups of `warps` warps, `groups` of them in a CTA.
struct LnShape {
    int64_t rows;
    int d, warps, groups;
    float eps, inv_d;
};

// NV values of a row a thread, in NV / VEC pieces: piece q covers columns (q * 32 warps + t) VEC...
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(LN_FWD_THREADS, NV <= 8 ? 6 : NV <= 16 ? 5 : NV <= 32 ? 4 : 2)
    ln_forward_kernel(LnShape s, const T* x, const void* w, const void* b, bool wf32, int form, T* y, float* mean,
                      float* rstd) {
    typedef typename Lanes<VEC>::V V;
    constexpr int NP = NV / VEC, N = Lanes<VEC>::N;
    __shared__ float red[2][LN_FWD_THREADS / 32];
    griddep_wait();
    griddep_launch();
    const int tpr = s.warps * 32, t = threadIdx.x % tpr, group = threadIdx.x / tpr, lane = threadIdx.x & 31;
    const int step = tpr * VEC, c0 = t * VEC;
    const int np = c0 < s.d ? min(NP, (s.d - c0 + step - 1) / step) : 0;  // this thread's pieces
    int flip = 0;
    auto row_sum = [&](float a) {
        a = warp_sum(a);
        if (s.warps == 1) return a;
        float* r = red[flip] + group * s.warps;  // the two halves in turn: one barrier a sum is enough
        flip ^= 1;
        if (lane == 0) r[t >> 5] = a;
        named_bar_sync(1 + group, tpr);
        a = 0.f;
        for (int i = 0; i < s.warps; ++i) a += r[i];
        return a;
    };
    for (int64_t r = (int64_t)blockIdx.x * s.groups + group; r < s.rows; r += (int64_t)gridDim.x * s.groups) {
        const T* xr = x + r * s.d + c0;
        Pack<T, VEC> p[NP];
#pragma unroll
        for (int q = 0; q < NP; ++q)
            if (q < np) p[q] = *reinterpret_cast<const Pack<T, VEC>*>(xr + q * step);
        V f[N], acc[N];
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = both<V>(0.f);
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            if (q >= np) break;
            widen(p[q], f);
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = add_(acc[i], f[i]);
        }
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) a += total(acc[i]);
        const float mu = row_sum(a) * s.inv_d;
        const V neg = both<V>(-mu);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = both<V>(0.f);
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            if (q >= np) break;
            opaque(p[q]);
            widen(p[q], f);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                f[i] = add_(f[i], neg);
                acc[i] = fma_(f[i], f[i], acc[i]);
            }
        }
        a = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) a += total(acc[i]);
        const float rs = rsqrtf(fmaf(row_sum(a), s.inv_d, s.eps));
        const V vrs = both<V>(rs);
        T* yr = y + r * s.d + c0;
        auto finish = [&](auto form) {
            constexpr int W = decltype(form)::value;
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                if (q >= np) break;
                V wv[N], bv[N];
                weights<T, VEC, W>(w, wf32, 1.f, c0 + q * step, wv);
                weights<T, VEC, W>(b, wf32, 0.f, c0 + q * step, bv);
                opaque(p[q]);
                widen(p[q], f);
#pragma unroll
                for (int i = 0; i < N; ++i) f[i] = fma_(mul_(add_(f[i], neg), vrs), wv[i], bv[i]);
                *reinterpret_cast<Pack<T, VEC>*>(yr + q * step) = narrow<T, VEC>(f);
            }
        };
        if (form == LN_W_ANY) finish(Int<LN_W_ANY>());
        else if (form == LN_W_SAME) finish(Int<LN_W_SAME>());
        else finish(Int<LN_W_F32>());
        if (t == 0) {
            if (mean) mean[r] = mu;
            if (rstd) rstd[r] = rs;
        }
    }
}

// Rows a group takes at a time: 32 values a thread, 16 where a value takes a register of its own.
__host__ __device__ constexpr int bwd_rows(size_t size, int vec, int nv) {
    return nv == 32 ? 1 : (vec == 1 || size == 4 ? 16 : 32) / nv;
}

// R rows at a time, NV columns a thread.
template <typename T, int VEC, int NV, int SLOTS>
__global__ void __launch_bounds__(LN_BWD_MOST, 1)
    ln_backward_kernel(LnShape s, const T* dy, const T* x, const void* w, bool wf32, const float* mean,
                       const float* rstd, T* dx, float* part) {
    typedef typename Lanes<VEC>::V V;
    constexpr int NP = NV / VEC, N = Lanes<VEC>::N, R = bwd_rows(sizeof(T), VEC, NV);
    __shared__ float red[2][16 * 2 * R];
    extern __shared__ __align__(16) uint8_t ln_smem[];
    float* const sums = reinterpret_cast<float*>(ln_smem);  // at the end, [2][d]: the CTA's partial sums
    griddep_wait();
    griddep_launch();
    const int tpr = s.warps * 32, t = threadIdx.x % tpr, group = threadIdx.x / tpr, lane = threadIdx.x & 31;
    const int step = tpr * VEC, c0 = t * VEC;
    const int np = c0 < s.d ? min(NP, (s.d - c0 + step - 1) / step) : 0;
    V wv[NP][N], dw[NP][N], db[NP][N];
#pragma unroll
    for (int q = 0; q < NP; ++q) {
#pragma unroll
        for (int i = 0; i < N; ++i) wv[q][i] = dw[q][i] = db[q][i] = both<V>(0.f);
        if (c0 + q * step < s.d) weights<T, VEC, LN_W_ANY>(w, wf32, 1.f, c0 + q * step, wv[q]);
    }
    // Pieces travel through SLOTS slots of shared memory by cp.async, a batch of rows a slot. A thread
    // copies the pieces that it reads itself, so no barrier guards the slots; 2-byte pieces are loaded
    // directly. Groups take R consecutive rows at a time; rows past the end are left out.
    constexpr bool ASYNC = sizeof(Pack<T, VEC>) >= 4;
    Pack<T, VEC>* const slot = reinterpret_cast<Pack<T, VEC>*>(ln_smem) + threadIdx.x;
    const int threads = blockDim.x, slot_pieces = 2 * R * NP * threads;
    const int64_t first = ((int64_t)blockIdx.x * s.groups + group) * R, stride = (int64_t)gridDim.x * s.groups * R;
    const int64_t hop = stride * s.d;
    const T *ax = x + first * s.d + c0, *ay = dy + first * s.d + c0;  // of the batch to be issued next
    int64_t ar = first;
    auto issue_rows = [&](int stage, auto rows) {
        Pack<T, VEC>* to = slot + stage * slot_pieces;
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (j >= rows) break;
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                if (q >= np) break;
                const int o = j * s.d + q * step;
                copy_async<sizeof(Pack<T, VEC>)>(to + 2 * (j * NP + q) * threads, ax + o);
                copy_async<sizeof(Pack<T, VEC>)>(to + (2 * (j * NP + q) + 1) * threads, ay + o);
            }
        }
    };
    auto issue = [&](int stage) {
        if (!ASYNC) return;
        if (ar + R <= s.rows) issue_rows(stage, R);
        else if (ar < s.rows) issue_rows(stage, (int)(s.rows - ar));
        asm volatile("cp.async.commit_group;" ::: "memory");
        ar += stride;
        ax += hop;
        ay += hop;
    };
    // the batch's statistics: lane j holds row j's mean, lane R + j its rstd
    auto stats = [&](int64_t r0) {
        const int j = lane % R;
        return lane < 2 * R && r0 + j < s.rows ? (lane < R ? mean : rstd)[r0 + j] : 0.f;
    };
    int flip = 0, stage = 0;
    for (int k = 0; k < SLOTS - 1; ++k) issue(k);
    float next = stats(first);
    for (int64_t r0 = first; r0 < s.rows; r0 += stride) {
        issue(stage == 0 ? SLOTS - 1 : stage - 1);
        float mu[R], rs[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            mu[j] = __shfl_sync(0xffffffffu, next, j);
            rs[j] = __shfl_sync(0xffffffffu, next, R + j);
        }
        next = stats(r0 + stride);
        const int rows = s.rows - r0 < R ? (int)(s.rows - r0) : R;
        const int64_t at = r0 * s.d + c0;
        Pack<T, VEC> px[R][NP], py[R][NP];
        if (ASYNC) asm volatile("cp.async.wait_group %0;" ::"n"(SLOTS - 1) : "memory");
        const Pack<T, VEC>* from = slot + stage * slot_pieces;
        auto take = [&](int rows, int np) {
#pragma unroll
            for (int j = 0; j < R; ++j) {
#pragma unroll
                for (int q = 0; q < NP; ++q) {
                    if (j < rows && q < np) {
                        if (ASYNC) {
                            px[j][q] = from[2 * (j * NP + q) * threads];
                            py[j][q] = from[(2 * (j * NP + q) + 1) * threads];
                        } else {
                            px[j][q] = *reinterpret_cast<const Pack<T, VEC>*>(x + at + (j * s.d + q * step));
                            py[j][q] = *reinterpret_cast<const Pack<T, VEC>*>(dy + at + (j * s.d + q * step));
                        }
                    } else {
                        memset(&px[j][q], 0, sizeof(px[j][q]));
                        memset(&py[j][q], 0, sizeof(py[j][q]));
                    }
                }
            }
        };
        if (rows == R && np == NP) take(R, NP);
        else take(rows, np);
        if (++stage == SLOTS) stage = 0;
        float v[2 * R];
        V xh[R][NP][N], g[R][NP][N];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const V neg = both<V>(-mu[j]), vrs = both<V>(rs[j]);
            V a = both<V>(0.f), b = both<V>(0.f);
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                widen(px[j][q], xh[j][q]);
                widen(py[j][q], g[j][q]);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    V &h = xh[j][q][i], &e = g[j][q][i];
                    h = mul_(add_(h, neg), vrs);
                    dw[q][i] = fma_(e, h, dw[q][i]);
                    db[q][i] = add_(db[q][i], e);
                    e = mul_(e, wv[q][i]);
                    a = add_(a, e);
                    b = fma_(e, h, b);
                }
            }
            v[2 * j] = total(a);
            v[2 * j + 1] = total(b);
        }
        float c[2 * R];
        const float mine = warp_sums<2 * R>(v, lane);
        if (s.warps == 1) {
#pragma unroll
            for (int i = 0; i < 2 * R; ++i) c[i] = __shfl_sync(0xffffffffu, mine, i * (16 / R)) * s.inv_d;
        } else {
            // [value][warp]; a lane adds every (16 / R)-th warp of its value, then those lanes add up
            constexpr int S = 16 / R;
            float* sh = red[flip] + group * s.warps * 2 * R;
            flip ^= 1;
            if (lane % S == 0) sh[(lane / S) * s.warps + (t >> 5)] = mine;
            named_bar_sync(1 + group, tpr);
            float a = 0.f;
            for (int k = lane % S; k < s.warps; k += S) a += sh[(lane / S) * s.warps + k];
#pragma unroll
            for (int o = S / 2; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
#pragma unroll
            for (int i = 0; i < 2 * R; ++i) c[i] = __shfl_sync(0xffffffffu, a, i * S) * s.inv_d;
        }
        T* out = dx + at;
        auto give = [&](int rows, int np) {
#pragma unroll
            for (int j = 0; j < R; ++j) {
                if (j >= rows) break;
                const V vrs = both<V>(rs[j]), c1 = both<V>(-c[2 * j]), c2 = both<V>(-c[2 * j + 1]);
#pragma unroll
                for (int q = 0; q < NP; ++q) {
                    if (q >= np) break;
                    V o[N];
#pragma unroll
                    for (int i = 0; i < N; ++i) o[i] = mul_(vrs, fma_(xh[j][q][i], c2, add_(g[j][q][i], c1)));
                    *reinterpret_cast<Pack<T, VEC>*>(out + (j * s.d + q * step)) = narrow<T, VEC>(o);
                }
            }
        };
        if (rows == R && np == NP) give(R, NP);
        else give(rows, np);
    }
    if (!part) return;
    // the groups' sums one after another in shared memory, so that the order is the same every time
    if (s.groups > 1) __syncthreads();
    float* pw = part + (size_t)blockIdx.x * 2 * s.d;
    for (int k = 0; k < s.groups; ++k) {
        if (group == k) {
            float* to = s.groups == 1 ? pw : sums;
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                if (c0 + q * step >= s.d) break;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int c = c0 + q * step + i;
                    const float* fw = reinterpret_cast<const float*>(&dw[q][0]);
                    const float* fb = reinterpret_cast<const float*>(&db[q][0]);
                    to[c] = k ? to[c] + fw[i] : fw[i];
                    to[s.d + c] = k ? to[s.d + c] + fb[i] : fb[i];
                }
            }
        }
        if (s.groups > 1) __syncthreads();
    }
    if (s.groups > 1)
        for (int c = threadIdx.x; c < 2 * s.d; c += blockDim.x) pw[c] = sums[c];
}

// dw (blockIdx.y 0) and db (1) from the CTAs' partial sums [parts][2][d].
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
    if (c < d) {
        const float* from = part + (size_t)blockIdx.y * d + c;
        for (int q = row; q < parts; q += 8 * LN_RED_ROWS) {  // eight loads in flight
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = q + k * LN_RED_ROWS < parts ? from[(size_t)(q + k * LN_RED_ROWS) * 2 * d] : 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) a += v[k];
        }
    }
    acc[row][lane] = a;
    __syncthreads();
    if (row || c >= d || !out) return;
    a = 0.f;
#pragma unroll
    for (int q = 0; q < LN_RED_ROWS; ++q) a += acc[q][lane];
    if (wf32) static_cast<float*>(out)[c] = a;
    else put(static_cast<T*>(out)[c], a);
}

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
    for (int v = (int)(16 / size); v > 1; v = v > 2 ? 2 : 1)
        if (c.d % v == 0 && aligned(a, v * size) && aligned(b, v * size) && aligned(e, v * size)) return v;
    return 1;
}

// Groups of `warps` warps in CTAs of about `threads` threads.
LnShape shape_of(const moe_layernorm_config& c, int warps, int threads) {
    LnShape s;
    s.rows = c.rows;
    s.d = c.d;
    s.eps = c.eps;
    s.inv_d = 1.0f / (float)c.d;
    s.warps = warps;
    s.groups = warps * 32 < threads ? threads / (warps * 32) : 1;
    return s;
}
int warps_for(int d, int values) { return (d + 32 * values - 1) / (32 * values); }

// f(Pack<T, VEC>) for the config's type and piece width.
template <typename F>
cudaError_t dispatch(int dtype, int vec, F f) {
    if (dtype == MOE_DTYPE_F32)
        return vec == 4 ? f(Pack<float, 4>()) : vec == 2 ? f(Pack<float, 2>()) : f(Pack<float, 1>());
    if (dtype == MOE_DTYPE_BF16)
        return vec == 8   ? f(Pack<__nv_bfloat16, 8>())
               : vec == 2 ? f(Pack<__nv_bfloat16, 2>())
                          : f(Pack<__nv_bfloat16, 1>());
    return vec == 8 ? f(Pack<__half, 8>()) : vec == 2 ? f(Pack<__half, 2>()) : f(Pack<__half, 1>());
}

// Backward: columns a thread keeps, and with them the warps of a row and the CTAs of the launch.
// (8 rather than 16 between 2048 and 4096: 16384 x 4096 bf16 91 us against 110 us)
int backward_values(int d) { return d <= 4096 ? 8 : d <= 8192 ? 16 : 32; }
LnShape backward_shape(const moe_layernorm_config& c) {
    return shape_of(c, warps_for(c.d, backward_values(c.d)), LN_BWD_THREADS);
}
int64_t backward_ctas(const moe_layernorm_config& c, int vec, int sms) {
    const LnShape s = backward_shape(c);
    const int rows = s.groups * bwd_rows(dtype_size(c.dtype), vec, backward_values(c.d));  // rows a CTA takes at a time
    const int64_t n = (c.rows + rows - 1) / rows, most = (int64_t)sms * (s.warps * s.groups > 8 ? 1 : 2);
    return n < most ? n : most;
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
    // Values a thread holds: 32 in as many warps as the row takes (64 above 8192 columns); 16 or 8 for short
    // rows, and where there are too few rows to fill the device (16 warps a SM). 64 values were slower
    // (4575 x 6651 fp32: 111 us against 75 us; 1511 x 1969 fp32: 18 us against 10.6 us with 16), 128 in
    // whole vectors no faster (16384 x 4096 bf16: 59 us both).
    int values = c->d <= 32 * LN_FWD_THREADS ? 32 : 64;
    while (values > 8 && (c->d <= 32 * values / 2 || c->rows * warps_for(c->d, values) < 16 * di.sms) &&
           warps_for(c->d, values / 2) <= LN_FWD_THREADS / 32)
        values /= 2;
    const LnShape s = shape_of(*c, warps_for(c->d, values), LN_FWD_THREADS);
    const int64_t n = (c->rows + s.groups - 1) / s.groups, most = (int64_t)di.sms * 64;
    const dim3 grid((unsigned)(n < most ? n : most)), block(32 * s.warps * s.groups);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t err = dispatch(c->dtype, vec, [&](auto pk) {
        typedef decltype(pk) P;
        typedef std::remove_reference_t<decltype(pk.v[0])> T;
        constexpr int V = (int)(sizeof(P) / sizeof(T));
        const bool wf32 = c->wdtype == MOE_DTYPE_F32;
        const size_t piece = wf32 ? (V < 4 ? V : 4) * 4 : V * sizeof(T);
        const int form = !w || !b || !aligned(w, piece) || !aligned(b, piece) ? LN_W_ANY : wf32 ? LN_W_F32 : LN_W_SAME;
        auto go = [&](auto kernel) {
            return launch_k(kernel, grid, block, 0, st, true, s, static_cast<const T*>(x), w, b, wf32, form,
                            static_cast<T*>(y), mean, rstd);
        };
        return values == 8    ? go(ln_forward_kernel<T, V, 8>)
               : values == 16 ? go(ln_forward_kernel<T, V, 16>)
               : values == 32 ? go(ln_forward_kernel<T, V, 32>)
                              : go(ln_forward_kernel<T, V, 64>);
    });
    return err == cudaSuccess ? MOE_OK : cuda_fail(err, "layer norm launch");
}

MOE_API int moe_layernorm_workspace_size(const moe_layernorm_config* c, size_t* bytes) {
    clear_error();
    const int rc = check(c);
    if (rc) return rc;
    if (!bytes) return fail(MOE_ERR_ARG, "bytes is NULL");
    *bytes = (size_t)backward_ctas(*c, 1, LN_MAX_SMS) * 2 * c->d * 4;
    if (*bytes == 0) *bytes = 8;
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
    const LnShape s = backward_shape(*c);
    const int ctas = (int)backward_ctas(*c, vec, di.sms);
    float* part = nullptr;
    if (dw || db) {
        const size_t need = (size_t)ctas * 2 * c->d * 4;
        if (!ws) return fail(MOE_ERR_ARG, "workspace is NULL");
        if (!aligned(ws, 16)) return fail(MOE_ERR_ARG, "workspace must be 16-byte aligned");
        if (ws_bytes < need) return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
        part = static_cast<float*>(ws);
    }
    const bool wf32 = c->wdtype == MOE_DTYPE_F32;
    const int values = backward_values(c->d);
    const cudaError_t err = dispatch(c->dtype, vec, [&](auto pk) {
        typedef decltype(pk) P;
        typedef std::remove_reference_t<decltype(pk.v[0])> T;
        constexpr int V = (int)(sizeof(P) / sizeof(T));
        auto go = [&](auto columns, auto slots) {
            constexpr int NV = decltype(columns)::value, SLOTS = decltype(slots)::value;
            constexpr auto kernel = &ln_backward_kernel<T, V, NV, SLOTS>;
            // bytes of the slots for each thread; 2-byte pieces have none
            constexpr size_t each = sizeof(P) < 4 ? 0 : (size_t)SLOTS * 2 * bwd_rows(sizeof(T), V, NV) * (NV / V) * sizeof(P);
            static_assert(each * LN_BWD_MOST <= 224 * 1024, "slots of the largest CTA");
            const int threads = 32 * s.warps * s.groups;
            size_t smem = each * threads;
            if (s.groups > 1 && smem < (size_t)2 * c->d * 4) smem = (size_t)2 * c->d * 4;
            // (the partial sums of several groups are at most 8 KB: they share a CTA up to 1024 columns)
            const cudaError_t e0 = allow_smem<kernel>(each * LN_BWD_MOST > 8192 ? each * LN_BWD_MOST : 8192);
            if (e0 != cudaSuccess) return e0;
            return launch_k(kernel, dim3(ctas), dim3(threads), smem, st, true, s, static_cast<const T*>(dy),
                            static_cast<const T*>(x), w, wf32, mean, rstd, static_cast<T*>(dx), part);
        };
        // 96 KB of slots and two CTAs a SM up to 2048 columns, 192 KB for one CTA above
        typedef Int<sizeof(T) == 4 ? 1 : 3> Wide;
        const cudaError_t e1 = values == 8    ? go(Int<8>(), Int<3>())
                               : values == 16 ? go(Int<16>(), Int<3>())
                                              : go(Int<32>(), Wide());
        if (e1 != cudaSuccess || !part) return e1;
        return launch_k(ln_reduce_kernel<T>, dim3((c->d + LN_RED_COLS - 1) / LN_RED_COLS, 2),
                        dim3(LN_RED_COLS * LN_RED_ROWS), 0, st, true, (const float*)part, ctas, c->d, wf32, dw, db);
    });
    return err == cudaSuccess ? MOE_OK : cuda_fail(err, "layer norm backward launch");
}

}  // extern "C"
