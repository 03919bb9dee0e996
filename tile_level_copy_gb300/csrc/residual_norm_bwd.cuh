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
// Calls that run one behind the other, 16384 x 2048 bf16, fp32 weights: layer norms 92 us (4.4 TB/s, 64 % of a copy's rate),
// mean-square norms 71 us (84 %; 72 with a gate). Layer norms take 51 instructions
// a value at 128 registers, with which 16 warps fit a SM, fill 53 % of the issue slots. 3001 x 1411 fp16 with a gate for
// each 250 rows: 35 us, five rows a group of warps between the kernel's start and the gates' ends.
#pragma once

#include "residual_norm.cuh"

namespace moe {
namespace {

// CTAs on a SM
__host__ __device__ constexpr int rb_ctas(int threads) { return threads > 256 ? 1 : 2; }
constexpr size_t RB_SMEM_MOST = 224 * 1024;
template <typename C>
constexpr int RB_BATCH = C::NU < 8 ? 4 : 8;  // units whose loads are in flight together

// A thread's units of w2 and, behind all of those, of k in shared memory.
template <typename C, int THREADS>
struct RbPlaces {
    f2* at;
    __device__ __forceinline__ f2* w2(int j) const { return at + j * THREADS; }
    __device__ __forceinline__ f2* k(int j) const { return at + (C::NU + j) * THREADS; }
};
// A batch of units of a vector, from unit j0 on.
template <typename C>
struct RbUnits {
    float v[RB_BATCH<C>][2];
};
// Reads them (null, and beyond the row: `none`) and writes them, in 16-byte pieces where the vector's alignment allows
// (`whole`). With a gate for every row single values bound the pass: a warp's lie 16 or 32 bytes apart (16384 x 2048
// bf16, mean-square norms: 254 us; in pieces 217).
template <typename T, typename C>
__device__ __forceinline__ RbUnits<C> vector_units(const C& c, const void* p, bool f32, bool whole, float none, int64_t at, int j0) {
    RbUnits<C> o;
    auto single = [&](auto value) {
#pragma unroll
        for (int k = 0; k < RB_BATCH<C>; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) o.v[k][i] = c.inside(j0 + k, i) ? value(at + c.column(j0 + k, i)) : none;
    };
    auto pieces = [&](auto from) {  // of type F
        typedef std::remove_const_t<std::remove_pointer_t<decltype(from)>> F;
#pragma unroll
        for (int k = 0; k < RB_BATCH<C>; k += C::UN) {
            const int q = (j0 + k) / C::UN;
            Pack<F, C::PV> e;
            if (q < c.np) {
#pragma unroll
                for (int n = 0; n < (int)sizeof(e) / 16; ++n)
                    reinterpret_cast<uint4*>(&e)[n] = reinterpret_cast<const uint4*>(from + (at + c.c0 + q * C::STEP))[n];
            }
#pragma unroll
            for (int n = 0; n < C::UN; ++n) {
                const float2 f = split(unit_of(e, n));
                o.v[k + n][0] = q < c.np ? f.x : none;
                o.v[k + n][1] = q < c.np ? f.y : none;
            }
        }
    };
    if (!p) {
        single([&](int64_t) { return none; });
        return o;
    }
    if constexpr (C::VEC > 1) {
        if (whole) {
            if (f32) pieces(static_cast<const float*>(p));
            else pieces(static_cast<const T*>(p));
            return o;
        }
    }
    if (f32) single([&](int64_t i) { return static_cast<const float*>(p)[i]; });
    else single([&](int64_t i) { return num(static_cast<const T*>(p)[i]); });
    return o;
}
template <typename T, typename C>
__device__ __forceinline__ void put_units(const C& c, void* p, bool f32, bool whole, int64_t at, int j0, const RbUnits<C>& o) {
    auto pieces = [&](auto to) {
        typedef std::remove_pointer_t<decltype(to)> F;
#pragma unroll
        for (int k = 0; k < RB_BATCH<C>; k += C::UN) {
            const int q = (j0 + k) / C::UN;
            Pack<F, C::PV> e;
#pragma unroll
            for (int n = 0; n < C::UN; ++n) put_unit(e, n, pair(o.v[k + n][0], o.v[k + n][1]));
            if (q >= c.np) continue;
#pragma unroll
            for (int n = 0; n < (int)sizeof(e) / 16; ++n)
                reinterpret_cast<uint4*>(to + (at + c.c0 + q * C::STEP))[n] = reinterpret_cast<const uint4*>(&e)[n];
        }
    };
    if constexpr (C::VEC > 1) {
        if (whole) {
            if (f32) pieces(static_cast<float*>(p));
            else pieces(static_cast<T*>(p));
            return;
        }
    }
#pragma unroll
    for (int k = 0; k < RB_BATCH<C>; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (!c.inside(j0 + k, i)) continue;
            const int64_t to = at + c.column(j0 + k, i);
            if (f32) static_cast<float*>(p)[to] = o.v[k][i];
            else put(static_cast<T*>(p)[to], o.v[k][i]);
        }
}
// Writes k of the rows that share gate g and, where its places hold something else, w2; zeros beyond the row. The sum
// of the thread's k. (This and gate_end are calls, made once a gate: inlined they took registers from the loop over the
// rows.)
template <typename T, typename C, typename Q>
__device__ __noinline__ float make_weights(const C c, const Q places, const RnWeights& w, int64_t g, bool with_w2) {
    static_assert(C::NU % RB_BATCH<C> == 0 && RB_BATCH<C> % C::UN == 0, "whole batches of whole pieces");
    float sum = 0.f;
#pragma unroll 1
    for (int j0 = 0; j0 < C::NU; j0 += RB_BATCH<C>) {
        RbUnits<C> a, k = vector_units<T>(c, w.post_w, w.f32, w.whole, 1.f, 0, j0);
        const RbUnits<C> gate = vector_units<T>(c, w.gate, w.f32, w.whole, 1.f, g * c.d, j0);
        if (with_w2) a = vector_units<T>(c, w.pre_w, w.f32, w.whole, 1.f, 0, j0);
#pragma unroll
        for (int n = 0; n < RB_BATCH<C>; ++n) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool in = c.inside(j0 + n, i);
                a.v[n][i] = in ? a.v[n][i] : 0.f;
                k.v[n][i] = in ? k.v[n][i] * gate.v[n][i] : 0.f;
                sum += k.v[n][i];
            }
            if (with_w2) *places.w2(j0 + n) = pair(a.v[n][0], a.v[n][1]);
            *places.k(j0 + n) = pair(k.v[n][0], k.v[n][1]);
        }
    }
    return sum;
}
// The end of the rows that share gate g: S lies in the places of k, B in those of w2. dw1 += gate S and db1 += gate B
// in sums [2][d] (fresh: nothing is there yet; last: they go to the places of k and w2), and w1 S + b1 B to part (a gate whose other rows lie elsewhere) or into dgate.
template <typename T, bool FULL, typename C, typename Q>
__device__ __noinline__ void gate_end(const C c, const Q places, const RnWeights& w, int64_t g, float* sums, float* part,
                                      void* dgate, bool whole_dgate, bool fresh, bool last) {
#pragma unroll 1
    for (int j0 = 0; j0 < C::NU; j0 += RB_BATCH<C>) {
        const RbUnits<C> gate = vector_units<T>(c, w.gate, w.f32, w.whole, 1.f, g * c.d, j0);
        const RbUnits<C> w1 = vector_units<T>(c, w.post_w, w.f32, w.whole, 1.f, 0, j0);
        RbUnits<C> a = vector_units<T>(c, fresh ? nullptr : sums, true, true, 0.f, 0, j0), b1, e, out;
        if (FULL) {
            b1 = vector_units<T>(c, w.post_b, w.f32, w.whole, 0.f, 0, j0);
            e = vector_units<T>(c, fresh ? nullptr : sums, true, true, 0.f, c.d, j0);
        }
#pragma unroll
        for (int k = 0; k < RB_BATCH<C>; ++k) {
            const float2 x = split(*places.k(j0 + k)), y = split(*places.w2(j0 + k));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float xs = i ? x.y : x.x, ys = i ? y.y : y.x;
                a.v[k][i] = fmaf(gate.v[k][i], xs, a.v[k][i]);
                out.v[k][i] = w1.v[k][i] * xs;
                if (FULL) {
                    e.v[k][i] = fmaf(gate.v[k][i], ys, e.v[k][i]);
                    out.v[k][i] = fmaf(b1.v[k][i], ys, out.v[k][i]);
                }
            }
        }
        if (last) {
#pragma unroll
            for (int k = 0; k < RB_BATCH<C>; ++k) {
                *places.k(j0 + k) = pair(a.v[k][0], a.v[k][1]);
                if (FULL) *places.w2(j0 + k) = pair(e.v[k][0], e.v[k][1]);
            }
        } else {
            put_units<T>(c, sums, true, true, 0, j0, a);
            if (FULL) put_units<T>(c, sums, true, true, c.d, j0, e);
        }
        if (!dgate) continue;
        if (part) put_units<T>(c, part, true, true, 0, j0, out);
        else put_units<T>(c, dgate, w.f32, whole_dgate, g * c.d, j0, out);
    }
}

// THREADS: at most so many in a CTA, and the stride of a thread's places in shared memory, so that they have fixed
// distances. Rows that are not there count as zeros, a norm that is not there as one with mean 0 and rstd 1 whose
// sums are left out: the same instructions serve every kind. GROUPED: more gates than one (a kernel of its own: the calls
// at a gate's end take registers from the loop over the rows).
template <typename T, int VEC, int NV, int THREADS, bool FULL, int MODE, bool GROUPED>
__global__ void __launch_bounds__(THREADS, rb_ctas(THREADS)) rn_backward_kernel(RnShape s, RnWeights w, RnBackward b) {
    typedef RnColumns<T, VEC, NV> C;
    typedef typename C::P P;
    typedef f2 V;
    constexpr int NP = C::NP, UN = C::UN, NU = C::NU, K = FULL ? 8 : 4, A = FULL ? 7 : 3;
    constexpr int NEXT = MODE == RN_OWN ? NV * THREADS * (int)sizeof(T) : rn_cover<T>(NV, THREADS);  // from tensor to tensor, bytes
    constexpr int SLOT = 4 * NEXT;
    __shared__ float red[2][THREADS / 32 * K];
    extern __shared__ __align__(16) uint8_t rb_smem[];
    griddep_wait();
    griddep_launch();
    const int tpr = s.warps * 32, t = threadIdx.x % tpr, group = threadIdx.x / tpr, lane = threadIdx.x & 31;
    const C cols(t, s.d);
    const bool post = s.post != 0;
    const T* const rows[4] = {static_cast<const T*>(b.dz), static_cast<const T*>(b.h), static_cast<const T*>(b.dh),
                              static_cast<const T*>(b.u)};
    const int64_t worker = (int64_t)blockIdx.x * s.groups + group, first = worker * s.chunk;
    const int total_rows = first < s.rows ? (int)(s.rows - first < s.chunk ? s.rows - first : s.chunk) : 0;

    const RbPlaces<C, THREADS> places{reinterpret_cast<V*>(rb_smem) + threadIdx.x};
    // A slot: the thread's pieces of the four tensors (own points at the first of them), or the 16-byte pieces that cover
    // the groups' rows.
    uint8_t* const own = rb_smem + 2 * NU * THREADS * sizeof(V) + (MODE == RN_OWN ? threadIdx.x * sizeof(P) : cover_at<T>(group, tpr, NV));
    // fetches row i of this worker, which starts at value `at` of the tensors
    auto issue = [&](int i, int64_t at, uint8_t* to) {
        if (MODE == RN_DIRECT) return;
        if (i < total_rows) {
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                if (!rows[n]) continue;
                if (MODE == RN_RAGGED) {
                    cover_row(to + n * NEXT, rows[n], s.rows * s.d, at, s.d, t, tpr);
                    continue;
                }
                const T* const from = rows[n] + (at + cols.c0);
#pragma unroll
                for (int q = 0; q < NP; ++q)
                    if (q < cols.np) copy_async<sizeof(P)>(to + n * NEXT + q * THREADS * sizeof(P), from + q * C::STEP);
            }
        }
        committed();
    };
    // Piece q of tensor n. Beyond the row and of tensors that are not there: zeros, which lie in the slots.
    auto take = [&](int n, const T* from, int q) {
        if (MODE == RN_OWN) return *reinterpret_cast<const P*>(reinterpret_cast<const uint8_t*>(from) + q * THREADS * sizeof(P));
        if constexpr (MODE == RN_RAGGED) return cols.load_padded(from, q);
        if (rows[n]) return cols.load(from, q);
        P p;
        memset(&p, 0, sizeof(p));
        return p;
    };

    const bool owner = MODE == RN_RAGGED && last_piece<T>(s.d) % tpr / 32 == t / 32;
    const bool next_owner = MODE == RN_RAGGED && (last_piece<T>(s.d) + 1) % tpr / 32 == t / 32;
    auto pad = [&](int64_t at, uint8_t* to) {
        __syncwarp();
#pragma unroll
        for (int n = 0; n < 4; ++n)
            if (rows[n]) pad_row(to + n * NEXT, rows[n], at, s.d, owner, next_owner, lane);
    };
    if (MODE == RN_RAGGED) {
        uint8_t* const slots = rb_smem + 2 * NU * THREADS * sizeof(V);
        for (int i = threadIdx.x * 16; i < s.slots * SLOT; i += blockDim.x * 16) *reinterpret_cast<uint4*>(slots + i) = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }
    if (MODE == RN_OWN) {
        P zero;
        memset(&zero, 0, sizeof(zero));
        for (int n = 0; n < 4; ++n)
            for (int k = 0; k < s.slots; ++k)
                for (int q = rows[n] ? cols.np : 0; q < NP; ++q)
                    *reinterpret_cast<P*>(own + k * SLOT + n * NEXT + q * THREADS * sizeof(P)) = zero;
    }
    int64_t at = first * s.d;
    for (int k = 0; k < s.slots - 1; ++k) issue(k, at + (int64_t)k * s.d, own + k * SLOT);
    const float2 plain = make_float2(0.f, 1.f);
    const float2 *const stats1 = post ? b.post_stats + first : nullptr, *const stats2 = s.pre ? b.pre_stats + first : nullptr;
    float2 next1 = post && total_rows ? stats1[0] : plain, next2 = s.pre && total_rows ? stats2[0] : plain;
    float ksum = 0.f;
    if (total_rows) {
        ksum = make_weights<T>(cols, places, w, GROUPED ? first / s.gate_rows : 0, true);
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
        if (GROUPED) {
            const int64_t left = s.gate_rows - (first + row) % s.gate_rows;
            if (left < stop - row) stop = row + (int)left;
        }
#pragma unroll 1
        for (; row < stop; ++row) {
            if (MODE == RN_RAGGED) {  // the row is there for all its threads, and they are done with the one before
                fetched(s.slots > 1 ? s.slots - 2 : 0);
                if (s.slots > 1) pad(at, here);
                named_bar_sync(1 + group, tpr);
            }
            issue(row + s.slots - 1, at + (int64_t)(s.slots - 1) * s.d, here == own ? own + (s.slots - 1) * SLOT : here - SLOT);
            if (MODE == RN_RAGGED && s.slots == 1) {
                fetched(0);
                pad(at, here);
                named_bar_sync(1 + group, tpr);
            }
            if (MODE == RN_OWN) fetched(s.slots - 1);
            const T* from[4];
#pragma unroll
            for (int n = 0; n < 4; ++n)
                from[n] = MODE == RN_DIRECT ? rows[n] + (at + cols.c0)
                                            : reinterpret_cast<const T*>(here + n * NEXT + (MODE == RN_RAGGED ? offset_of(rows[n] + at) + cols.c0 * (int)sizeof(T) : 0));
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
                    const P pz = take(0, from[0], q), ph = take(1, from[1], q), pd = take(2, from[2], q), pu = take(3, from[3], q);
#pragma unroll
                    for (int i = 0; i < UN; ++i) {
                        const int j = q * UN + i;
                        const V z = unit_of(pz, i), hn = fma_(unit_of(ph, i), rs2, neg2), gy = mul_(z, *places.w2(j));
                        const V e = fma_(rs2, gy, unit_of(pd, i)), k = *places.k(j), ku = mul_(k, fma_(unit_of(pu, i), rs1, neg1));
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
                const P pz = take(0, from[0], q), ph = take(1, from[1], q), pd = take(2, from[2], q), pu = take(3, from[3], q);
                P px, pv;
#pragma unroll
                for (int i = 0; i < UN; ++i) {
                    const int j = q * UN + i;
                    V dt = unit_of(pd, i);
                    if (FULL) dt = add_(dt, b1);
                    dt = fma_(unit_of(ph, i), a1, fma_(rs2, mul_(unit_of(pz, i), *places.w2(j)), dt));
                    put_unit(px, i, mul_(dt, res));
                    const V un = fma_(unit_of(pu, i), rs1, neg1);
                    s1[j] = fma_(dt, un, s1[j]);
                    if (FULL) s2[FULL ? j : 0] = add_(s2[FULL ? j : 0], dt);
                    V m = o3;  // (0 without a post norm: u may be infinite)
                    if (post) m = FULL ? fma_(un, o2, o3) : mul_(un, o2);
                    put_unit(pv, i, fma_(mul_(dt, *places.k(j)), o1, m));
                }
                cols.store(static_cast<T*>(b.dx) + (at + cols.c0), q, px);
                if (b.du) cols.store(static_cast<T*>(b.du) + (at + cols.c0), q, pv);
            }
            here = here == own + (s.slots - 1) * SLOT ? own : here + SLOT;
            at += s.d;
        }
        if (GROUPED) {
            // A gate whose rows all lie here is done; else these rows' sums: in the first row those of a gate that began
            // earlier or that the worker begins with. S and B pass through the weights' places.
            const int64_t g = (first + row - 1) / s.gate_rows;
            const bool whole = g * s.gate_rows >= first && (row < total_rows || (g + 1) * s.gate_rows <= first + row || first + row == s.rows);
            float* const p = b.gpart + (2 * worker + (g == first / s.gate_rows ? 0 : 1)) * s.d;
            const V branch = both<V>(s.branch);
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                *places.k(j) = mul_(s1[j], branch);
                if (FULL) *places.w2(j) = mul_(s2[FULL ? j : 0], branch);
                s1[j] = both<V>(0.f);
                if (FULL) s2[FULL ? j : 0] = both<V>(0.f);
            }
            if (b.part) gate_end<T, FULL>(cols, places, w, g, b.gsum + 2 * worker * s.d, whole ? nullptr : p, b.dgate,
                                          (reinterpret_cast<uintptr_t>(b.dgate) & 15) == 0, g == first / s.gate_rows, row == total_rows);
            if (row < total_rows) ksum = make_weights<T>(cols, places, w, g + 1, FULL);
        }
    }
    if (MODE != RN_DIRECT) fetched(0);
    if (!b.part) return;
    const V branch = both<V>(s.branch);
#pragma unroll
    for (int j = 0; j < NU; ++j) {
        if (!GROUPED) {
            s1[j] = mul_(s1[j], branch);
            if (FULL) s2[FULL ? j : 0] = mul_(s2[FULL ? j : 0], branch);
        } else if (total_rows) {  // dw1 and db1 in the place of S and B
            s1[j] = *places.k(j);
            if (FULL) s2[FULL ? j : 0] = *places.w2(j);
        }
    }
    // the groups' sums side by side in shared memory, then added up in the order of the groups
    constexpr int SUMS = FULL ? 4 : 2;
    float* const pw = b.part + (size_t)blockIdx.x * SUMS * s.d;
    float* const sums = reinterpret_cast<float*>(rb_smem);
    if (s.groups > 1) __syncthreads();
    float* const to = s.groups == 1 ? pw : sums + (size_t)group * SUMS * s.d;
#pragma unroll
    for (int j = 0; j < NU; ++j) {
#pragma unroll
        for (int n = 0; n < SUMS; ++n) {
            const V v = n == 0 ? sp[j] : n == SUMS / 2 ? s1[j] : n == 1 ? sq[FULL ? j : 0] : s2[FULL ? j : 0];
            if constexpr (VEC > 1) {
                if (cols.inside(j, 0)) *reinterpret_cast<V*>(to + n * s.d + cols.column(j, 0)) = v;
            } else {
                const float2 e = split(v);
                if (cols.inside(j, 0)) to[n * s.d + cols.column(j, 0)] = e.x;
                if (cols.inside(j, 1)) to[n * s.d + cols.column(j, 1)] = e.y;
            }
        }
    }
    if (s.groups == 1) return;
    __syncthreads();
    for (int c = threadIdx.x; c < SUMS * s.d; c += blockDim.x) {
        float a = 0.f;
        for (int k = 0; k < s.groups; ++k) a += sums[k * SUMS * s.d + c];
        pw[c] = a;
    }
}

}  // namespace

template <typename T>
cudaError_t launch_residual_backward(RnShape s, const RnWeights& w, const RnBackward& b, int vec, bool full, bool grouped,
                                     int ctas, cudaStream_t st) {
    const int threads = 32 * s.warps * s.groups;
    auto launch = [&](auto width, auto values, auto most, auto whole, auto how, auto gates) {
        constexpr int VEC = decltype(width)::value, NV = decltype(values)::value, THREADS = decltype(most)::value;
        constexpr int MODE = decltype(how)::value;
        constexpr auto kernel = &rn_backward_kernel<T, VEC, NV, THREADS, decltype(whole)::value, MODE, decltype(gates)::value>;
        constexpr size_t weights = (size_t)2 * NV * THREADS * 4, row = (size_t)4 * NV * THREADS * sizeof(T);
        constexpr size_t slot = MODE == RN_DIRECT ? 0 : MODE == RN_OWN ? row : (size_t)4 * rn_cover<T>(NV, THREADS);
        constexpr size_t room = RB_SMEM_MOST / rb_ctas(THREADS);
        static_assert(weights + slot <= RB_SMEM_MOST, "room for a row");
        s.slots = MODE == RN_DIRECT ? 1 : weights + 3 * slot <= room ? 3 : weights + 2 * slot <= room ? 2 : 1;
        size_t smem = weights + s.slots * slot;
        const size_t sums = (size_t)(full ? 4 : 2) * s.d * 4 * s.groups;  // of every group, at the end
        if (s.groups > 1 && smem < sums) smem = sums;
        const cudaError_t e = allow_smem<kernel>(RB_SMEM_MOST);
        if (e != cudaSuccess) return e;
        return launch_k(kernel, dim3(ctas), dim3(threads), smem, st, true, s, w, b);
    };
    auto go = [&](auto width, auto values, auto most, auto whole, auto how) {
        return grouped ? launch(width, values, most, whole, how, std::true_type()) : launch(width, values, most, whole, how, std::false_type());
    };
    auto kinds = [&](auto width, auto values, auto most, auto how) {
        return full ? go(width, values, most, std::true_type(), how) : go(width, values, most, std::false_type(), how);
    };
    constexpr int VEC = 16 / sizeof(T);
    typedef Int<RN_OWN> Own;
    typedef Int<RN_RAGGED> Ragged;
    typedef Int<RN_DIRECT> Direct;
    const bool one = vec == 1;
    if (full && (grouped || sizeof(T) == 4) && s.d <= 2048) {
        auto short_rows = [&](auto gates) {
            return one ? launch(Int<1>(), Int<8>(), Int<256>(), std::true_type(), Ragged(), gates)
                       : launch(Int<VEC>(), Int<8>(), Int<256>(), std::true_type(), Own(), gates);
        };
        if (grouped) return short_rows(std::true_type());
        if constexpr (sizeof(T) == 4) return short_rows(std::false_type());
    }
    if (s.d > 8192)
        return one ? kinds(Int<1>(), Int<32>(), Int<512>(), Direct()) : kinds(Int<VEC>(), Int<32>(), Int<512>(), Direct());
    if (threads > 256) return one ? kinds(Int<1>(), Int<16>(), Int<512>(), Ragged()) : kinds(Int<VEC>(), Int<16>(), Int<512>(), Own());
    return one ? kinds(Int<1>(), Int<16>(), Int<256>(), Ragged()) : kinds(Int<VEC>(), Int<16>(), Int<256>(), Own());
}

}  // namespace moe
