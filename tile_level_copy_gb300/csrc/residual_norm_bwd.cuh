// Backward pass of the residual norm: dx, du and the CTAs' sums for the weights' gradients, in one pass over the rows.
//
//   hn = (h - mean2) rstd2, gy = dz w2, e = dh + rstd2 gy          un = (u - mean1) rstd1, k = gate w1
//   dt = e - rstd2 (sum(gy) + hn sum(gy hn)) / d                   (sum(gy) only where the norm takes the mean off)
//   dx = a dt,   du = c rstd1 (k dt - sum(k dt) / d - un sum(k un dt) / d)
//   dw2 += dz hn, db2 += dz, S += c dt un, B += c dt;  dw1 += gate S, db1 += gate B, dgate = w1 S + b1 B
//
// dt is linear in the first two sums, so the sums over it follow from sums over e, hn and un: one reduction and one
// barrier a row instead of two. HBM traffic bounds the pass: dz, dh, u, h are read, dx, du written. A thread keeps the
// same columns over all its rows, with the four sums of each in registers; a group of warps takes consecutive rows,
// which come through shared memory by cp.async while the rows before are worked on. w2 and k lie in shared memory in
// fp32. A thread reads and writes only its own places there, so no barrier guards them. S and B are those of the rows
// that share a gate: where these end, dgate is written and dw1 and db1, in the workspace, take them up. With one
// gate for all rows that happens after the CTAs' sums are added up. Rows above 8192 values are read from global memory
// twice: their slots would find no room beside the weights.
#pragma once

#include "residual_norm.cuh"

namespace moe {
namespace {

// CTAs on a SM
__host__ __device__ constexpr int rb_ctas(int, int threads) { return threads > 256 ? 1 : 2; }
constexpr size_t RB_SMEM_MOST = 224 * 1024;


// Two neighbouring values of a piece of 16-bit or 32-bit values, or its only one, as fp32; and back. (By words: pieces of
// two 16-bit values that are copied one by one cost a byte permutation each, a quarter of the kernel's instructions.)
template <typename T, int VEC>
__device__ __forceinline__ typename Lanes<VEC>::V unit_of(const Pack<T, VEC>& p, int j) {
    if constexpr (VEC == 1) {
        return num(p.v[0]);
    } else if constexpr (sizeof(T) == 4) {
        return pair(p.v[2 * j], p.v[2 * j + 1]);
    } else {
        const uint32_t w = reinterpret_cast<const uint32_t*>(&p)[j];
        if constexpr (std::is_same_v<T, __nv_bfloat16>) {
            return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
            return pair(f.x, f.y);
        }
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void put_unit(Pack<T, VEC>& p, int j, typename Lanes<VEC>::V v) {
    if constexpr (VEC == 1) {
        put(p.v[0], v);
    } else {
        const float2 f = split(v);
        if constexpr (sizeof(T) == 4) {
            p.v[2 * j] = f.x;
            p.v[2 * j + 1] = f.y;
        } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
            reinterpret_cast<uint32_t*>(&p)[j] = pack_bf16x2(f.x, f.y);
        } else {
            const __half2 h = __floats2half2_rn(f.x, f.y);
            reinterpret_cast<uint32_t*>(&p)[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
}

// Bytes of a tensor in a slot of ragged rows: the rows of up to eight groups, each with what covers its ends.
template <typename T>
__host__ __device__ constexpr int rb_cover(int values, int threads) { return values * threads * (int)sizeof(T) + 8 * 32; }
// Where a row's values start behind a 16-byte boundary.
__device__ __forceinline__ int offset_of(const void* p) { return (int)(reinterpret_cast<uintptr_t>(p) & 15); }
// Thread t of `threads` fetches its share of the 16-byte pieces that cover the d values from `at` on. A piece that
// reaches beyond the tensor's n values is copied value by value.
template <typename T>
__device__ __forceinline__ void cover_row(uint8_t* to, const T* rows, int64_t n, int64_t at, int d, int t, int threads) {
    const T* const from = rows + at;
    const int off = offset_of(from), pieces = (off + d * (int)sizeof(T) + 15) / 16;
    const uint8_t* const start = reinterpret_cast<const uint8_t*>(from) - off;
    const uint8_t *const lo = reinterpret_cast<const uint8_t*>(rows), *const hi = reinterpret_cast<const uint8_t*>(rows + n);
    for (int i = t; i < pieces; i += threads) {
        const uint8_t* const p = start + 16 * i;
        if (p >= lo && p + 16 <= hi) {
            copy_async<16>(to + 16 * i, p);
        } else {
            for (int k = 0; k < 16; k += (int)sizeof(T))
                if (p + k >= lo && p + k < hi) *reinterpret_cast<T*>(to + 16 * i + k) = *reinterpret_cast<const T*>(p + k);
        }
    }
}
// A thread's columns in units of U values, UN of them in a piece, `np` pieces in the row; and where its units of w2 and,
// behind all of those, of k lie in shared memory.
template <int U_, int UN_, int NU_, int THREADS_>
struct RbColumns {
    static constexpr int U = U_, UN = UN_, NU = NU_, THREADS = THREADS_;
    typedef typename Lanes<U>::V V;
    int c0, step, np, d;
    V* at;
    __device__ __forceinline__ int column(int j) const { return c0 + (j / UN) * step + (j % UN) * U; }
    __device__ __forceinline__ bool inside(int j) const { return j / UN < np; }
    __device__ __forceinline__ V* w2(int j) const { return at + j * THREADS; }
    __device__ __forceinline__ V* k(int j) const { return at + (NU + j) * THREADS; }
};
constexpr int RB_BATCH = 4;  // units whose loads are in flight together
template <typename T, typename C>
__device__ __forceinline__ void vector_units(const C& c, const void* p, bool f32, float none, int64_t at, int j0,
                                             Pack<float, C::U> (&o)[RB_BATCH]) {
    auto each = [&](auto value) {
#pragma unroll
        for (int k = 0; k < RB_BATCH; ++k)
#pragma unroll
            for (int i = 0; i < C::U; ++i) o[k].v[i] = c.inside(j0 + k) ? value(at + c.column(j0 + k) + i) : none;
    };
    if (!p) each([&](int64_t) { return none; });
    else if (f32) each([&](int64_t i) { return static_cast<const float*>(p)[i]; });
    else each([&](int64_t i) { return num(static_cast<const T*>(p)[i]); });
}
// Writes w2, and k of the rows that share gate g; zeros beyond the row. The sum of the thread's k. (This and
// gate_end are calls, made once a gate: inlined they took registers from the loop over the rows.)
template <typename T, typename C>
__device__ __noinline__ float make_weights(const C c, const RnWeights& w, int64_t g) {
    typedef typename C::V V;
    float sum = 0.f;
#pragma unroll 1
    for (int j0 = 0; j0 < C::NU; j0 += RB_BATCH) {
        Pack<float, C::U> a[RB_BATCH], k[RB_BATCH], gate[RB_BATCH];
        vector_units<T>(c, w.pre_w, w.f32, 1.f, 0, j0, a);
        vector_units<T>(c, w.post_w, w.f32, 1.f, 0, j0, k);
        vector_units<T>(c, w.gate, w.f32, 1.f, g * c.d, j0, gate);
#pragma unroll
        for (int n = 0; n < RB_BATCH; ++n) {
#pragma unroll
            for (int i = 0; i < C::U; ++i) {
                a[n].v[i] = c.inside(j0 + n) ? a[n].v[i] : 0.f;
                k[n].v[i] = c.inside(j0 + n) ? k[n].v[i] * gate[n].v[i] : 0.f;
                sum += k[n].v[i];
            }
            *c.w2(j0 + n) = *reinterpret_cast<const V*>(&a[n]);
            *c.k(j0 + n) = *reinterpret_cast<const V*>(&k[n]);
        }
    }
    return sum;
}
// The end of the rows that share gate g: S lies in the places of k, B in those of w2. dw1 += gate S and db1 += gate B
// in sums [2][d], and w1 S + b1 B to part (a gate whose other rows lie elsewhere) or into dgate.
template <typename T, bool FULL, typename C>
__device__ __noinline__ void gate_end(const C c, const RnWeights& w, int64_t g, float* sums, float* part, void* dgate) {
    typedef typename C::V V;
#pragma unroll 1
    for (int j0 = 0; j0 < C::NU; j0 += RB_BATCH) {
        Pack<float, C::U> gate[RB_BATCH], w1[RB_BATCH], b1[RB_BATCH];
        V a[RB_BATCH], e[RB_BATCH];
        vector_units<T>(c, w.gate, w.f32, 1.f, g * c.d, j0, gate);
        vector_units<T>(c, w.post_w, w.f32, 1.f, 0, j0, w1);
        if (FULL) vector_units<T>(c, w.post_b, w.f32, 0.f, 0, j0, b1);
        auto at = [&](int n, int k) { return reinterpret_cast<V*>(sums + (int64_t)n * c.d + c.column(j0 + k)); };
#pragma unroll
        for (int k = 0; k < RB_BATCH; ++k) {
            if (!c.inside(j0 + k)) continue;
            a[k] = *at(0, k);
            if (FULL) e[k] = *at(1, k);
        }
#pragma unroll
        for (int k = 0; k < RB_BATCH; ++k) {
            if (!c.inside(j0 + k)) continue;
            const V x = *c.k(j0 + k), y = *c.w2(j0 + k), gt = *reinterpret_cast<const V*>(&gate[k]);
            *at(0, k) = fma_(gt, x, a[k]);
            if (FULL) *at(1, k) = fma_(gt, y, e[k]);
            if (!dgate) continue;
            V o = mul_(*reinterpret_cast<const V*>(&w1[k]), x);
            if (FULL) o = fma_(*reinterpret_cast<const V*>(&b1[k]), y, o);
#pragma unroll
            for (int i = 0; i < C::U; ++i) {
                const int col = c.column(j0 + k) + i;
                const float out = reinterpret_cast<const float*>(&o)[i];
                if (part) part[col] = out;
                else if (w.f32) static_cast<float*>(dgate)[g * c.d + col] = out;
                else put(static_cast<T*>(dgate)[g * c.d + col], out);
            }
        }
    }
}

// How rows reach their readers. RB_OWN: a thread fetches the pieces that it reads itself, so no barrier guards the slots.
// RB_RAGGED: rows of odd addresses, whose values only 2-byte or 4-byte loads could fetch one by one: the threads of a row
// fetch the 16-byte pieces that cover it and read single values from them, one barrier a row. RB_DIRECT: values are
// read from global memory in both passes over them (rows too wide for a slot).
enum RbMode : int { RB_OWN, RB_RAGGED, RB_DIRECT };

// THREADS: at most so many in a CTA, and the stride of a thread's places in shared memory, so that they have fixed
// distances. Rows that are not there count as zeros, a norm that is not there as one with mean 0 and rstd 1 whose
// sums are left out: the same instructions serve every kind.
template <typename T, int VEC, int NV, int THREADS, bool FULL, int MODE>
__global__ void __launch_bounds__(THREADS, rb_ctas(NV, THREADS)) rn_backward_kernel(RnShape s, RnWeights w, RnBackward b, int grouped) {
    typedef typename Lanes<VEC>::V V;  // a unit: two values, or one
    typedef Pack<T, VEC> P;
    constexpr int U = VEC < 2 ? 1 : 2, NP = NV / VEC, UN = VEC / U, NU = NP * UN, K = FULL ? 8 : 4, A = FULL ? 7 : 3;
    constexpr int SLOT = MODE == RB_OWN ? 4 * NV * THREADS * (int)sizeof(T) : 4 * rb_cover<T>(NV, THREADS);  // bytes
    __shared__ float red[2][THREADS / 32 * K];
    extern __shared__ __align__(16) uint8_t rb_smem[];
    griddep_wait();
    griddep_launch();
    const int tpr = s.warps * 32, t = threadIdx.x % tpr, group = threadIdx.x / tpr, lane = threadIdx.x & 31;
    const int step = tpr * VEC, c0 = t * VEC;
    const int np = c0 < s.d ? min(NP, (s.d - c0 + step - 1) / step) : 0;
    const bool post = s.post != 0;
    const T* const rows[4] = {static_cast<const T*>(b.dz), static_cast<const T*>(b.h), static_cast<const T*>(b.dh),
                              static_cast<const T*>(b.u)};
    const int64_t worker = (int64_t)blockIdx.x * s.groups + group, first = worker * s.chunk;
    const int total_rows = first < s.rows ? (int)(s.rows - first < s.chunk ? s.rows - first : s.chunk) : 0;

    // this thread's units of w2 and of k
    V* const wsm = reinterpret_cast<V*>(rb_smem) + threadIdx.x;
    const RbColumns<U, UN, NU, THREADS> cols{c0, step, np, s.d, wsm};
    // A slot: the thread's pieces of the four tensors (own points at the first of them), or the 16-byte pieces that cover
    // the groups' rows.
    uint8_t* const slots = rb_smem + 2 * NU * THREADS * sizeof(V);
    uint8_t* const own = slots + (MODE == RB_OWN ? threadIdx.x * sizeof(P) : group * (tpr * NV * (int)sizeof(T) + 32));
    constexpr int NEXT = MODE == RB_OWN ? NP * THREADS * (int)sizeof(P) : rb_cover<T>(NV, THREADS);  // from tensor to tensor
    // fetches row i of this worker, whose first value of the thread is value `at` of the tensors
    auto issue = [&](int i, int64_t at, uint8_t* to) {
        if (MODE == RB_DIRECT) return;
        if (i < total_rows) {
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                if (!rows[n]) continue;
                if (MODE == RB_RAGGED) {
                    cover_row(to + n * NEXT, rows[n], s.rows * s.d, at - c0, s.d, t, tpr);
                    continue;
                }
                const T* const from = rows[n] + at;
#pragma unroll
                for (int q = 0; q < NP; ++q)
                    if (q < np) fetch(reinterpret_cast<P*>(to + n * NEXT + q * THREADS * sizeof(P)), reinterpret_cast<const P*>(from + q * step));
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // Piece q of tensor n. Beyond the row and of tensors that are not there: zeros, which lie in the slots.
    auto take = [&](int n, const uint8_t* here, int64_t at, int q) {
        P p;
        if (MODE == RB_OWN) {
            p = *reinterpret_cast<const P*>(here + n * NEXT + q * THREADS * sizeof(P));
        } else {
            memset(&p, 0, sizeof(p));
            if (rows[n] && q < np) {
                if (MODE == RB_DIRECT) p = *reinterpret_cast<const P*>(rows[n] + at + q * step);
                else p = *reinterpret_cast<const P*>(here + n * NEXT + offset_of(rows[n] + (at - c0)) + (c0 + q * step) * (int)sizeof(T));
            }
        }
        return p;
    };

    if (MODE == RB_OWN) {
        P zero;
        memset(&zero, 0, sizeof(zero));
        for (int n = 0; n < 4; ++n)
            for (int k = 0; k < s.slots; ++k)
                for (int q = rows[n] ? np : 0; q < NP; ++q)
                    *reinterpret_cast<P*>(own + k * SLOT + n * NEXT + q * THREADS * sizeof(P)) = zero;
    }
    int64_t at = first * s.d + c0;
    for (int k = 0; k < s.slots - 1; ++k) issue(k, at + (int64_t)k * s.d, own + k * SLOT);
    const float2 plain = make_float2(0.f, 1.f);
    const float2 *const stats1 = post ? b.post_stats + first : nullptr, *const stats2 = s.pre ? b.pre_stats + first : nullptr;
    float2 next1 = post && total_rows ? stats1[0] : plain, next2 = s.pre && total_rows ? stats2[0] : plain;
    float ksum = 0.f;
    if (total_rows) {
        ksum = make_weights<T>(cols, w, grouped ? first / s.gate_rows : 0);
        if (grouped && b.part) {
            float* const sums = b.gsum + 2 * worker * s.d;
            for (int j = 0; j < np * UN; ++j) {
                *reinterpret_cast<V*>(sums + cols.column(j)) = both<V>(0.f);
                if (FULL) *reinterpret_cast<V*>(sums + s.d + cols.column(j)) = both<V>(0.f);
            }
        }
    }
    // sums of a thread's columns: dw2, db2, S / c, B / c
    V sp[NU], sq[FULL ? NU : 1], s1[NU], s2[FULL ? NU : 1];
#pragma unroll
    for (int j = 0; j < NU; ++j) {
        sp[j] = s1[j] = both<V>(0.f);
        if (FULL) sq[FULL ? j : 0] = s2[FULL ? j : 0] = both<V>(0.f);
    }

    const V res = both<V>(s.res);
    int flip = 0;
    uint8_t* here = own;
    // rows that share a gate; what a gate's end takes stays out of the loop over them
    for (int row = 0; row < total_rows;) {
        int stop = total_rows;
        if (grouped) {
            const int64_t left = s.gate_rows - (first + row) % s.gate_rows;
            if (left < stop - row) stop = row + (int)left;
        }
#pragma unroll 1
        for (; row < stop; ++row) {
            if (MODE == RB_RAGGED) {  // the row is there for all its threads, and they are done with the one before
                fetched(s.slots > 1 ? s.slots - 2 : 0);
                named_bar_sync(1 + group, tpr);
            }
            issue(row + s.slots - 1, at + (int64_t)(s.slots - 1) * s.d, here == own ? own + (s.slots - 1) * SLOT : here - SLOT);
            if (MODE == RB_RAGGED && s.slots == 1) {
                fetched(0);
                named_bar_sync(1 + group, tpr);
            }
            if (MODE == RB_OWN) fetched(s.slots - 1);
            const V neg1 = both<V>(-next1.x * next1.y), rs1 = both<V>(next1.y), rs2 = both<V>(next2.y);
            const float rstd1 = next1.y, rstd2 = next2.y, off2 = -next2.x * next2.y;
            if (row + 1 < total_rows) {
                if (post) next1 = stats1[row + 1];
                if (s.pre) next2 = stats2[row + 1];
            }
            float v[K];
            {
                const V neg2 = both<V>(off2);
                V a[A];
#pragma unroll
                for (int i = 0; i < A; ++i) a[i] = both<V>(0.f);
#pragma unroll
                for (int q = 0; q < NP; ++q) {
                    const P pz = take(0, here, at, q), ph = take(1, here, at, q), pd = take(2, here, at, q), pu = take(3, here, at, q);
#pragma unroll
                    for (int i = 0; i < UN; ++i) {
                        const int j = q * UN + i;
                        const V z = unit_of(pz, i), hn = fma_(unit_of(ph, i), rs2, neg2), gy = mul_(z, *cols.w2(j));
                        const V e = fma_(rs2, gy, unit_of(pd, i)), k = *cols.k(j), ku = mul_(k, fma_(unit_of(pu, i), rs1, neg1));
                        sp[j] = fma_(z, hn, sp[j]);
                        a[0] = fma_(gy, hn, a[0]);
                        a[1] = fma_(ku, e, a[1]);
                        a[2] = fma_(ku, hn, a[2]);
                        if (FULL) {
                            sq[FULL ? j : 0] = add_(sq[FULL ? j : 0], z);
                            a[FULL ? 3 : 0] = add_(a[FULL ? 3 : 0], gy);
                            a[FULL ? 4 : 0] = fma_(k, e, a[FULL ? 4 : 0]);
                            a[FULL ? 5 : 0] = add_(a[FULL ? 5 : 0], ku);
                            a[FULL ? 6 : 0] = fma_(k, hn, a[FULL ? 6 : 0]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < K; ++i) v[i] = i < A ? total(a[i < A ? i : 0]) : ksum;
            }
            // sums over the row: warp by shuffles, warps through shared memory, [value][warp]
            float c[K];
            const float mine = warp_sums<K>(v, lane);
            constexpr int S = 32 / K;
            if (s.warps == 1) {
#pragma unroll
                for (int i = 0; i < K; ++i) c[i] = __shfl_sync(0xffffffffu, mine, i * S);
            } else {
                float* sh = red[flip] + group * s.warps * K;
                flip ^= 1;
                if (lane % S == 0) sh[(lane / S) * s.warps + (t >> 5)] = mine;
                named_bar_sync(1 + group, tpr);
                float a = 0.f;
                for (int k = lane % S; k < s.warps; k += S) a += sh[(lane / S) * s.warps + k];
#pragma unroll
                for (int o = S / 2; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
#pragma unroll
                for (int i = 0; i < K; ++i) c[i] = __shfl_sync(0xffffffffu, a, i * S);
            }
            // dt = e - p0 - hn p1; m0, m1: the sums of k dt and of k un dt
            const float p1 = s.pre ? rstd2 * c[0] * s.inv_d : 0.f;
            const float p0 = FULL && s.pre == MOE_NORM_LAYER ? rstd2 * c[FULL ? 3 : 0] * s.inv_d : 0.f;
            float m1 = post ? c[1] - p1 * c[2] : 0.f, m0 = 0.f;
            if (FULL) {
                if (post) m1 -= p0 * c[FULL ? 5 : 0];
                if (s.post == MOE_NORM_LAYER) m0 = c[FULL ? 4 : 0] - p0 * c[FULL ? 7 : 0] - p1 * c[FULL ? 6 : 0];
            }
            // dt = dh + b1 + rstd2 gy + a1 h, du = o1 k dt + o2 un + o3
            const float scale = s.branch * rstd1, back = -scale * s.inv_d;
            const V a1 = both<V>(-p1 * rstd2), b1 = both<V>(-p1 * off2 - p0);
            const V o1 = both<V>(scale), o2 = both<V>(back * m1), o3 = both<V>(back * m0);
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                const P pz = take(0, here, at, q), ph = take(1, here, at, q), pd = take(2, here, at, q), pu = take(3, here, at, q);
                P px, pv;
#pragma unroll
                for (int i = 0; i < UN; ++i) {
                    const int j = q * UN + i;
                    V dt = unit_of(pd, i);
                    if (FULL) dt = add_(dt, b1);
                    dt = fma_(unit_of(ph, i), a1, fma_(rs2, mul_(unit_of(pz, i), *cols.w2(j)), dt));
                    put_unit(px, i, mul_(dt, res));
                    const V un = fma_(unit_of(pu, i), rs1, neg1);
                    s1[j] = fma_(dt, un, s1[j]);
                    if (FULL) s2[FULL ? j : 0] = add_(s2[FULL ? j : 0], dt);
                    V m = o3;  // (0 without a post norm: u may be infinite)
                    if (post) m = FULL ? fma_(un, o2, o3) : mul_(un, o2);
                    put_unit(pv, i, fma_(mul_(dt, *cols.k(j)), o1, m));
                }
                if (q < np) {
                    *reinterpret_cast<P*>(static_cast<T*>(b.dx) + at + q * step) = px;
                    if (b.du) *reinterpret_cast<P*>(static_cast<T*>(b.du) + at + q * step) = pv;
                }
            }
            here = here == own + (s.slots - 1) * SLOT ? own : here + SLOT;
            at += s.d;
        }
        if (grouped) {
            // A gate whose rows all lie here is done; else these rows' sums: in the first row those of a gate that began
            // earlier or that the worker begins with. S and B pass through the weights' places.
            const int64_t g = (first + row - 1) / s.gate_rows;
            const bool whole = g * s.gate_rows >= first && (row < total_rows || (g + 1) * s.gate_rows <= first + row || first + row == s.rows);
            float* const p = b.gpart + (2 * worker + (g == first / s.gate_rows ? 0 : 1)) * s.d;
            const V branch = both<V>(s.branch);
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                *cols.k(j) = mul_(s1[j], branch);
                if (FULL) *cols.w2(j) = mul_(s2[FULL ? j : 0], branch);
                s1[j] = both<V>(0.f);
                if (FULL) s2[FULL ? j : 0] = both<V>(0.f);
            }
            if (b.part) gate_end<T, FULL>(cols, w, g, b.gsum + 2 * worker * s.d, whole ? nullptr : p, b.dgate);
            if (row < total_rows) ksum = make_weights<T>(cols, w, g + 1);
        }
    }
    if (MODE != RB_DIRECT) fetched(0);
    if (!b.part) return;
    const V branch = both<V>(s.branch);
#pragma unroll
    for (int j = 0; j < NU; ++j) {
        if (!grouped) {
            s1[j] = mul_(s1[j], branch);
            if (FULL) s2[FULL ? j : 0] = mul_(s2[FULL ? j : 0], branch);
        } else if (total_rows && cols.inside(j)) {  // dw1 and db1 in the place of S and B
            const float* const sums = b.gsum + 2 * worker * s.d + cols.column(j);
            s1[j] = *reinterpret_cast<const V*>(sums);
            if (FULL) s2[FULL ? j : 0] = *reinterpret_cast<const V*>(sums + s.d);
        }
    }
    // the groups' sums one after another in shared memory, so that the order is the same every time
    constexpr int SUMS = FULL ? 4 : 2;
    float* const sums = reinterpret_cast<float*>(rb_smem);
    float* const pw = b.part + (size_t)blockIdx.x * SUMS * s.d;
    if (s.groups > 1) __syncthreads();
    for (int k = 0; k < s.groups; ++k) {
        if (group == k) {
            float* to = s.groups == 1 ? pw : sums;
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                if (!cols.inside(j)) break;
#pragma unroll
                for (int n = 0; n < SUMS; ++n) {
                    const V v = n == 0 ? sp[j] : n == SUMS / 2 ? s1[j] : n == 1 ? sq[FULL ? j : 0] : s2[FULL ? j : 0];
                    V* const p = reinterpret_cast<V*>(to + n * s.d + cols.column(j));  // d is a multiple of the unit
                    *p = k ? add_(*p, v) : v;
                }
            }
        }
        if (s.groups > 1) __syncthreads();
    }
    if (s.groups > 1)
        for (int c = threadIdx.x; c < SUMS * s.d; c += blockDim.x) pw[c] = sums[c];
}

}  // namespace

template <typename T>
cudaError_t launch_residual_backward(const RnShape& shape, const RnWeights& w, const RnBackward& b, int vec, bool full,
                                     bool grouped, int ctas, cudaStream_t st) {
    RnShape s = shape;
    const int threads = 32 * s.warps * s.groups, values = rn_backward_values(s.d);
    auto go = [&](auto width, auto columns, auto most, auto whole, auto how) {
        constexpr int VEC = decltype(width)::value, NV = decltype(columns)::value, THREADS = decltype(most)::value;
        constexpr int MODE = decltype(how)::value;
        constexpr auto kernel = &rn_backward_kernel<T, VEC, NV, THREADS, decltype(whole)::value, MODE>;
        constexpr size_t weights = (size_t)2 * NV * THREADS * 4;
        constexpr size_t slot = MODE == RB_DIRECT ? 0 : MODE == RB_OWN ? (size_t)4 * NV * THREADS * sizeof(T) : (size_t)4 * rb_cover<T>(NV, THREADS);
        constexpr size_t room = RB_SMEM_MOST / rb_ctas(NV, THREADS);
        static_assert(weights + slot <= RB_SMEM_MOST, "room for a row");
        s.slots = MODE == RB_DIRECT ? 1 : weights + 3 * slot <= room ? 3 : weights + 2 * slot <= room ? 2 : 1;
        size_t smem = weights + s.slots * slot;
        if (s.groups > 1 && smem < (size_t)(full ? 4 : 2) * s.d * 4) smem = (size_t)(full ? 4 : 2) * s.d * 4;
        const cudaError_t e = allow_smem<kernel>(RB_SMEM_MOST);
        if (e != cudaSuccess) return e;
        return launch_k(kernel, dim3(ctas), dim3(threads), smem, st, true, s, w, b, (int)grouped);
    };
    auto kinds = [&](auto width, auto columns, auto most, auto how) {
        return full ? go(width, columns, most, std::true_type(), how) : go(width, columns, most, std::false_type(), how);
    };
    constexpr int VEC = 16 / sizeof(T);
    typedef Int<RB_OWN> Own;
    typedef Int<RB_RAGGED> Ragged;
    typedef Int<RB_DIRECT> Direct;
    const bool one = vec == 1;
    if (values == 32) return one ? kinds(Int<1>(), Int<32>(), Int<512>(), Direct()) : kinds(Int<VEC>(), Int<32>(), Int<512>(), Direct());
    if (threads > 256) return one ? kinds(Int<1>(), Int<16>(), Int<512>(), Ragged()) : kinds(Int<VEC>(), Int<16>(), Int<512>(), Own());
    return one ? kinds(Int<1>(), Int<16>(), Int<256>(), Ragged()) : kinds(Int<VEC>(), Int<16>(), Int<256>(), Own());
}

}  // namespace moe
