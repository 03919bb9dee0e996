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
__host__ __device__ constexpr int rb_ctas(int values, int threads) { return threads > 256 ? 1 : values == 8 ? 3 : 2; }
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

// DIRECT: rows are read from global memory in both passes over them (2-byte pieces, rows too wide for a slot).
// THREADS: at most so many in a CTA, and the stride of a thread's places in shared memory, so that they have fixed
// distances. Rows that are not there count as zeros, a norm that is not there as one with mean 0 and rstd 1 whose
// sums are left out: the same instructions serve every kind.
template <typename T, int VEC, int NV, int THREADS, bool FULL, bool DIRECT>
__global__ void __launch_bounds__(THREADS, rb_ctas(NV, THREADS)) rn_backward_kernel(RnShape s, RnWeights w, RnBackward b, int grouped) {
    typedef typename Lanes<VEC>::V V;  // a unit: two values, or one
    typedef Pack<T, VEC> P;
    constexpr int U = VEC < 2 ? 1 : 2, NP = NV / VEC, UN = VEC / U, NU = NP * UN, K = FULL ? 8 : 4, A = FULL ? 7 : 3;
    typedef Pack<float, U> F;
    __shared__ float red[2][THREADS / 32 * K];
    extern __shared__ __align__(16) uint8_t rb_smem[];
    griddep_wait();
    griddep_launch();
    const int tpr = s.warps * 32, t = threadIdx.x % tpr, group = threadIdx.x / tpr, lane = threadIdx.x & 31;
    const int step = tpr * VEC, c0 = t * VEC;
    const int np = c0 < s.d ? min(NP, (s.d - c0 + step - 1) / step) : 0;
    const bool pre = s.pre != 0, post = s.post != 0, lay1 = s.post == MOE_NORM_LAYER, lay2 = s.pre == MOE_NORM_LAYER;
    const T* const rows[4] = {static_cast<const T*>(b.dz), static_cast<const T*>(b.h), static_cast<const T*>(b.dh),
                              static_cast<const T*>(b.u)};
    T *const dx = static_cast<T*>(b.dx), *const du = static_cast<T*>(b.du);
    const int64_t worker = (int64_t)blockIdx.x * s.groups + group;
    const int64_t first = worker * s.chunk, last = first + s.chunk < s.rows ? first + s.chunk : s.rows;

    // this thread's units of w2 and of k
    V* const wsm = reinterpret_cast<V*>(rb_smem) + threadIdx.x;
    auto at_w2 = [&](int j) { return wsm + j * THREADS; };
    auto at_k = [&](int j) { return wsm + (NU + j) * THREADS; };
    auto column = [&](int j) { return c0 + (j / UN) * step + (j % UN) * U; };
    // with a gate for each group of rows: dw1 and db1 so far
    auto at_sum = [&](int n, int j) { return reinterpret_cast<V*>(b.gsum + (2 * worker + n) * s.d + column(j)); };
    // a slot: pieces of the four tensors
    P* const slots = reinterpret_cast<P*>(rb_smem + 2 * NU * THREADS * sizeof(V)) + threadIdx.x;
    auto piece = [&](int stage, int tensor, int q) { return slots + stage * (4 * NP * THREADS) + (tensor * NP + q) * THREADS; };
    auto issue = [&](int64_t r, int stage) {
        if (DIRECT) return;
        if (r < last) {
            const int64_t at = r * s.d + c0;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                if (!rows[n]) continue;
#pragma unroll
                for (int q = 0; q < NP; ++q) {
                    if (q >= np) break;
                    fetch(piece(stage, n, q), reinterpret_cast<const P*>(rows[n] + at + q * step));
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto take = [&](int n, int stage, int64_t at, int q) {
        if (!DIRECT) return *piece(stage, n, q);
        P p;
        if (rows[n]) p = *reinterpret_cast<const P*>(rows[n] + at + q * step);
        else memset(&p, 0, sizeof(p));
        return p;
    };
    // w2, and k of the rows that share gate g; the sum of this thread's k
    float ksum = 0.f;
    auto make_w = [&](int64_t g) {
        ksum = 0.f;
#pragma unroll 1
        for (int j = 0; j < np * UN; ++j) {
            F f, k;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int col = column(j) + i;
                f.v[i] = value_at<T>(w.pre_w, w.f32, col, 1.f);
                k.v[i] = value_at<T>(w.post_w, w.f32, col, 1.f) * value_at<T>(w.gate, w.f32, g * s.d + col, 1.f);
                ksum += k.v[i];
            }
            *at_w2(j) = *reinterpret_cast<const V*>(&f);
            *at_k(j) = *reinterpret_cast<const V*>(&k);
        }
    };

    if (!DIRECT) {
        P zero;
        memset(&zero, 0, sizeof(zero));
        for (int n = 0; n < 4; ++n)
            if (!rows[n])
                for (int k = 0; k < s.slots; ++k)
                    for (int q = 0; q < NP; ++q) *piece(k, n, q) = zero;
    }
    int flip = 0, stage = 0;
    for (int k = 0; k < s.slots - 1; ++k) issue(first + k, k);
    const float2 plain = make_float2(0.f, 1.f);
    float2 next1 = post && first < last ? b.post_stats[first] : plain, next2 = pre && first < last ? b.pre_stats[first] : plain;
    int64_t g = 0, g_end = s.rows;  // the row's gate and where its rows end
    if (grouped && first < last) {
        g = first / s.gate_rows;
        g_end = (g + 1) * s.gate_rows;
    }
    const int64_t g0 = g;
    if (first < last) {
        make_w(g);
        if (grouped && b.part) {
#pragma unroll 1
            for (int j = 0; j < np * UN; ++j) {
                *at_sum(0, j) = both<V>(0.f);
                if (FULL) *at_sum(1, j) = both<V>(0.f);
            }
        }
    }
    // sums of a thread's columns: dw2, db2, S, B
    V sp[NU], sq[FULL ? NU : 1], s1[NU], s2[FULL ? NU : 1];
#pragma unroll
    for (int j = 0; j < NU; ++j) {
        sp[j] = s1[j] = both<V>(0.f);
        if (FULL) sq[FULL ? j : 0] = s2[FULL ? j : 0] = both<V>(0.f);
    }

    const V branch = both<V>(s.branch), res = both<V>(s.res);
    for (int64_t r = first; r < last; ++r) {
        issue(r + s.slots - 1, stage == 0 ? s.slots - 1 : stage - 1);
        const float2 st1 = next1, st2 = next2;
        if (post && r + 1 < last) next1 = b.post_stats[r + 1];
        if (pre && r + 1 < last) next2 = b.pre_stats[r + 1];
        if (!DIRECT) fetched(s.slots - 1);
        const int64_t at = r * s.d + c0;
        const V neg1 = both<V>(-st1.x * st1.y), rs1 = both<V>(st1.y), neg2 = both<V>(-st2.x * st2.y), rs2 = both<V>(st2.y);
        float v[K];
        {
            V a[A];
#pragma unroll
            for (int i = 0; i < A; ++i) a[i] = both<V>(0.f);
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                if (q >= np) break;
                const P pz = take(0, stage, at, q), ph = take(1, stage, at, q), pd = take(2, stage, at, q), pu = take(3, stage, at, q);
#pragma unroll
                for (int i = 0; i < UN; ++i) {
                    const int j = q * UN + i;
                    const V z = unit_of(pz, i), hn = fma_(unit_of(ph, i), rs2, neg2), gy = mul_(z, *at_w2(j));
                    const V e = fma_(rs2, gy, unit_of(pd, i)), k = *at_k(j), ku = mul_(k, fma_(unit_of(pu, i), rs1, neg1));
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
        const float p1 = pre ? st2.y * c[0] * s.inv_d : 0.f, p0 = FULL && lay2 ? st2.y * c[FULL ? 3 : 0] * s.inv_d : 0.f;
        float m1 = post ? c[1] - p1 * c[2] : 0.f, m0 = 0.f;
        if (FULL) {
            if (post) m1 -= p0 * c[FULL ? 5 : 0];
            if (lay1) m0 = c[FULL ? 4 : 0] - p0 * c[FULL ? 7 : 0] - p1 * c[FULL ? 6 : 0];
        }
        const V n0 = both<V>(-p0), n1 = both<V>(-p1), k0 = both<V>(-m0 * s.inv_d), k1 = both<V>(-m1 * s.inv_d);
        const V out1 = both<V>(s.branch * st1.y);
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            if (q >= np) break;
            const P pz = take(0, stage, at, q), ph = take(1, stage, at, q), pd = take(2, stage, at, q), pu = take(3, stage, at, q);
            P px, pv;
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                const int j = q * UN + i;
                const V hn = fma_(unit_of(ph, i), rs2, neg2), gy = mul_(unit_of(pz, i), *at_w2(j));
                V e = fma_(rs2, gy, unit_of(pd, i));
                if (FULL) e = add_(e, n0);
                e = fma_(hn, n1, e);
                put_unit(px, i, mul_(e, res));
                const V un = fma_(unit_of(pu, i), rs1, neg1), d = mul_(e, branch);
                s1[j] = fma_(d, un, s1[j]);
                if (FULL) s2[FULL ? j : 0] = add_(s2[FULL ? j : 0], d);
                V m = k0;  // (0 without a post norm: u may be infinite)
                if (post) m = FULL ? fma_(un, k1, k0) : mul_(un, k1);
                put_unit(pv, i, mul_(fma_(e, *at_k(j), m), out1));
            }
            *reinterpret_cast<P*>(dx + at + q * step) = px;
            if (du) *reinterpret_cast<P*>(du + at + q * step) = pv;
        }
        if (++stage == s.slots) stage = 0;
        if (grouped && (r + 1 == g_end || r + 1 == last)) {
            // a gate whose rows all lie here is done; else these rows' sums: the first gate's in the first row.
            // S and B pass through the weights' places, so that what follows need not be unrolled
            const bool whole = g * s.gate_rows >= first && (g_end <= last || last == s.rows);
            float* const p = b.gpart + (2 * worker + (g == g0 ? 0 : 1)) * s.d;
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                if (j / UN >= np) break;
                *at_k(j) = s1[j];
                if (FULL) *at_w2(j) = s2[FULL ? j : 0];
                s1[j] = both<V>(0.f);
                if (FULL) s2[FULL ? j : 0] = both<V>(0.f);
            }
#pragma unroll 1
            for (int j = 0; b.part && j < np * UN; ++j) {
                F x, y, a, e;
                *reinterpret_cast<V*>(&x) = *at_k(j);
                *reinterpret_cast<V*>(&a) = *at_sum(0, j);
                if (FULL) {
                    *reinterpret_cast<V*>(&y) = *at_w2(j);
                    *reinterpret_cast<V*>(&e) = *at_sum(1, j);
                }
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int col = column(j) + i;
                    const float gate = value_at<T>(w.gate, w.f32, g * s.d + col, 1.f);
                    a.v[i] = fmaf(gate, x.v[i], a.v[i]);
                    if (FULL) e.v[i] = fmaf(gate, y.v[i], e.v[i]);
                    if (b.dgate) {
                        float out = value_at<T>(w.post_w, w.f32, col, 1.f) * x.v[i];
                        if (FULL) out = fmaf(value_at<T>(w.post_b, w.f32, col, 0.f), y.v[i], out);
                        if (!whole) p[col] = out;
                        else if (w.f32) static_cast<float*>(b.dgate)[g * s.d + col] = out;
                        else put(static_cast<T*>(b.dgate)[g * s.d + col], out);
                    }
                }
                *at_sum(0, j) = *reinterpret_cast<const V*>(&a);
                if (FULL) *at_sum(1, j) = *reinterpret_cast<const V*>(&e);
            }
            if (r + 1 < last) {
                ++g;
                g_end += s.gate_rows;
                make_w(g);
            }
        }
    }
    if (!DIRECT) fetched(0);
    if (!b.part) return;
    if (grouped && first < last) {  // dw1 and db1 in the place of S and B
#pragma unroll
        for (int j = 0; j < NU; ++j) {
            if (j / UN >= np) break;
            s1[j] = *at_sum(0, j);
            if (FULL) s2[FULL ? j : 0] = *at_sum(1, j);
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
                if (j / UN >= np) break;
#pragma unroll
                for (int n = 0; n < SUMS; ++n) {
                    const V v = n == 0 ? sp[j] : n == SUMS / 2 ? s1[j] : n == 1 ? sq[FULL ? j : 0] : s2[FULL ? j : 0];
                    V* const p = reinterpret_cast<V*>(to + n * s.d + column(j));  // d is a multiple of the unit
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
    auto go = [&](auto width, auto columns, auto most, auto whole, auto straight) {
        constexpr int VEC = decltype(width)::value, NV = decltype(columns)::value, THREADS = decltype(most)::value;
        constexpr bool DIRECT = decltype(straight)::value;
        constexpr auto kernel = &rn_backward_kernel<T, VEC, NV, THREADS, decltype(whole)::value, DIRECT>;
        constexpr size_t weights = (size_t)2 * NV * THREADS * 4, slot = DIRECT ? 0 : (size_t)4 * NV * THREADS * sizeof(T);
        constexpr size_t room = RB_SMEM_MOST / rb_ctas(NV, THREADS);
        static_assert(weights + slot <= RB_SMEM_MOST, "room for a row");
        s.slots = DIRECT ? 1 : weights + 3 * slot <= room ? 3 : weights + 2 * slot <= room ? 2 : 1;
        size_t smem = weights + s.slots * slot;
        if (s.groups > 1 && smem < (size_t)(full ? 4 : 2) * s.d * 4) smem = (size_t)(full ? 4 : 2) * s.d * 4;
        const cudaError_t e = allow_smem<kernel>(RB_SMEM_MOST);
        if (e != cudaSuccess) return e;
        return launch_k(kernel, dim3(ctas), dim3(threads), smem, st, true, s, w, b, (int)grouped);
    };
    auto kinds = [&](auto width, auto columns, auto most, auto straight) {
        return full ? go(width, columns, most, std::true_type(), straight) : go(width, columns, most, std::false_type(), straight);
    };
    constexpr int VEC = 16 / sizeof(T);
    typedef std::integral_constant<bool, (sizeof(T) < 4)> Two;  // 2-byte pieces cannot be fetched asynchronously
    const bool one = vec == 1;
    if (values == 32) return one ? kinds(Int<1>(), Int<32>(), Int<512>(), std::true_type()) : kinds(Int<VEC>(), Int<32>(), Int<512>(), std::true_type());
    if (threads > 256) return one ? kinds(Int<1>(), Int<16>(), Int<512>(), Two()) : kinds(Int<VEC>(), Int<16>(), Int<512>(), std::false_type());
    if (values == 16) return one ? kinds(Int<1>(), Int<16>(), Int<256>(), Two()) : kinds(Int<VEC>(), Int<16>(), Int<256>(), std::false_type());
    return one ? kinds(Int<1>(), Int<8>(), Int<256>(), Two()) : kinds(Int<VEC>(), Int<8>(), Int<256>(), std::false_type());
}

}  // namespace moe
