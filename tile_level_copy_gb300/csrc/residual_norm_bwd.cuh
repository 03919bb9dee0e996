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

constexpr int RB_MOST = 512;
constexpr size_t RB_SMEM_MOST = 224 * 1024;


// DIRECT: rows are read from global memory in both passes over them (2-byte pieces, rows too wide for a slot).
template <typename T, int VEC, int NV, bool FULL, bool DIRECT>
__global__ void __launch_bounds__(RB_MOST, 1) rn_backward_kernel(RnShape s, RnWeights w, RnBackward b, int grouped, int wbytes) {
    constexpr int U = VEC < 2 ? VEC : 2;  // values worked on at a time, a unit (4 spill more)
    typedef typename Lanes<U>::V V;
    typedef Pack<T, VEC> P;
    typedef Pack<float, U> F;
    constexpr int NP = NV / VEC, UN = VEC / U, NU = NP * UN, N = Lanes<U>::N, K = FULL ? 8 : 4;
    __shared__ float red[2][16 * K];
    extern __shared__ __align__(16) uint8_t rb_smem[];
    griddep_wait();
    griddep_launch();
    const int tpr = s.warps * 32, t = threadIdx.x % tpr, group = threadIdx.x / tpr, lane = threadIdx.x & 31;
    const int threads = blockDim.x, step = tpr * VEC, c0 = t * VEC;
    const int np = c0 < s.d ? min(NP, (s.d - c0 + step - 1) / step) : 0;
    const bool pre = s.pre != 0, post = s.post != 0, lay1 = s.post == MOE_NORM_LAYER, lay2 = s.pre == MOE_NORM_LAYER;
    const T *const gz = static_cast<const T*>(b.dz), *const gh = static_cast<const T*>(b.h);
    const T *const gd = static_cast<const T*>(b.dh), *const gu = static_cast<const T*>(b.u);
    T *const dx = static_cast<T*>(b.dx), *const du = static_cast<T*>(b.du);
    const int64_t worker = (int64_t)blockIdx.x * s.groups + group;
    const int64_t first = worker * s.chunk, last = first + s.chunk < s.rows ? first + s.chunk : s.rows;

    // this thread's units of w2 and of k
    F* const wsm = reinterpret_cast<F*>(rb_smem) + threadIdx.x;
    auto at_w2 = [&](int j) { return wsm + j * threads; };
    auto at_k = [&](int j) { return wsm + (NU + j) * threads; };
    auto column = [&](int j) { return c0 + (j / UN) * step + (j % UN) * U; };
    // with a gate for each group of rows: dw1 and db1 so far
    auto at_sum = [&](int n, int j) { return reinterpret_cast<F*>(b.gsum + (2 * worker + n) * s.d + column(j)); };
    // tensors in a slot, one behind the other: dz, h, dh, u, as far as they are there
    const int at_d = pre ? 2 : 0, at_u = at_d + (gd ? 1 : 0), tensors = at_u + (gu ? 1 : 0);
    P* const slot = reinterpret_cast<P*>(rb_smem + wbytes) + threadIdx.x;
    auto piece = [&](int stage, int tensor, int q) { return slot + ((stage * tensors + tensor) * s.pieces + q) * threads; };
    auto issue = [&](int64_t r, int stage) {
        if (DIRECT) return;
        if (r < last) {
            const int64_t at = r * s.d + c0;
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                if (q >= np) break;
                if (pre) {
                    fetch(piece(stage, 0, q), reinterpret_cast<const P*>(gz + at + q * step));
                    fetch(piece(stage, 1, q), reinterpret_cast<const P*>(gh + at + q * step));
                }
                if (gd) fetch(piece(stage, at_d, q), reinterpret_cast<const P*>(gd + at + q * step));
                if (gu) fetch(piece(stage, at_u, q), reinterpret_cast<const P*>(gu + at + q * step));
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto take = [&](const T* from, int stage, int tensor, int64_t at, int q) {
        return DIRECT ? *reinterpret_cast<const P*>(from + at + q * step) : *piece(stage, tensor, q);
    };
    auto unit = [](const P& p, int j) { return *reinterpret_cast<const Pack<T, U>*>(&p.v[j * U]); };
    // w2, and k of the rows that share gate g
    auto make_w = [&](int64_t g) {
#pragma unroll 1
        for (int j = 0; j < np * UN; ++j) {
            F f, k;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int col = column(j) + i;
                f.v[i] = value_at<T>(w.pre_w, w.f32, col, 1.f);
                k.v[i] = value_at<T>(w.post_w, w.f32, col, 1.f) * value_at<T>(w.gate, w.f32, g * s.d + col, 1.f);
            }
            *at_w2(j) = f;
            *at_k(j) = k;
        }
    };

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
                F zero;
#pragma unroll
                for (int i = 0; i < U; ++i) zero.v[i] = 0.f;
                *at_sum(0, j) = zero;
                if (FULL) *at_sum(1, j) = zero;
            }
        }
    }
    // sums of a thread's columns: dw2, db2, S, B
    V sp[NU][N], sq[FULL ? NU : 1][N], s1[NU][N], s2[FULL ? NU : 1][N];
#pragma unroll
    for (int j = 0; j < NU; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            sp[j][i] = s1[j][i] = both<V>(0.f);
            if (FULL) sq[FULL ? j : 0][i] = s2[FULL ? j : 0][i] = both<V>(0.f);
        }

    const V branch = both<V>(s.branch), res = both<V>(s.res);
    for (int64_t r = first; r < last; ++r) {
        issue(r + s.slots - 1, stage == 0 ? s.slots - 1 : stage - 1);
        const float2 st1 = next1, st2 = next2;
        if (post && r + 1 < last) next1 = b.post_stats[r + 1];
        if (pre && r + 1 < last) next2 = b.pre_stats[r + 1];
        if (!DIRECT) fetched(s.slots - 1);
        const int64_t at = r * s.d + c0;
        const V neg1 = both<V>(-st1.x), rs1 = both<V>(st1.y), neg2 = both<V>(-st2.x), rs2 = both<V>(st2.y);
        // e and hn of a unit, dz in z, gy = dz w2 in y
        auto above = [&](const P& pz, const P& ph, const P& pd, int j, V (&e)[N], V (&hn)[N], V (&z)[N], V (&y)[N]) {
            if (gd) {
                widen(unit(pd, j % UN), e);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) e[i] = both<V>(0.f);
            }
            if (pre) {
                widen(unit(ph, j % UN), hn);
                widen(unit(pz, j % UN), z);
                widen(*at_w2(j), y);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    hn[i] = mul_(add_(hn[i], neg2), rs2);
                    y[i] = mul_(z[i], y[i]);
                    e[i] = fma_(rs2, y[i], e[i]);
                }
            }
        };
        float v[K];
        {
            V a[K];
#pragma unroll
            for (int i = 0; i < K; ++i) a[i] = both<V>(0.f);
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                if (q >= np) break;
                P pz, ph, pd, pu;
                if (pre) {
                    pz = take(gz, stage, 0, at, q);
                    ph = take(gh, stage, 1, at, q);
                }
                if (gd) pd = take(gd, stage, at_d, at, q);
                if (post) pu = take(gu, stage, at_u, at, q);
#pragma unroll
                for (int j = q * UN; j < (q + 1) * UN; ++j) {
                    V e[N], hn[N], z[N], y[N];
                    above(pz, ph, pd, j, e, hn, z, y);
                    if (pre) {
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            sp[j][i] = fma_(z[i], hn[i], sp[j][i]);
                            a[0] = fma_(y[i], hn[i], a[0]);
                            if (FULL) {
                                sq[FULL ? j : 0][i] = add_(sq[FULL ? j : 0][i], z[i]);
                                a[3] = add_(a[3], y[i]);
                            }
                        }
                    }
                    if (post) {
                        V un[N], k[N];
                        widen(unit(pu, j % UN), un);
                        widen(*at_k(j), k);
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            const V ku = mul_(k[i], mul_(add_(un[i], neg1), rs1));
                            a[1] = fma_(ku, e[i], a[1]);
                            if (pre) a[2] = fma_(ku, hn[i], a[2]);
                            if (FULL) {
                                a[4] = fma_(k[i], e[i], a[4]);
                                a[5] = add_(a[5], k[i]);
                                a[6] = add_(a[6], ku);
                                if (pre) a[7] = fma_(k[i], hn[i], a[7]);
                            }
                        }
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < K; ++i) v[i] = total(a[i]);
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
        float m1 = c[1] - p1 * c[2], m0 = 0.f;
        if (FULL) {
            m1 -= p0 * c[FULL ? 6 : 0];
            if (lay1) m0 = c[FULL ? 4 : 0] - p0 * c[FULL ? 5 : 0] - p1 * c[FULL ? 7 : 0];
        }
        const V n0 = both<V>(-p0), n1 = both<V>(-p1), k0 = both<V>(-m0 * s.inv_d), k1 = both<V>(-m1 * s.inv_d);
        const V out1 = both<V>(s.branch * st1.y);
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            if (q >= np) break;
            P pz, ph, pd, pu, px;
            if (pre) {
                pz = take(gz, stage, 0, at, q);
                ph = take(gh, stage, 1, at, q);
            }
            if (gd) pd = take(gd, stage, at_d, at, q);
            if (gu) pu = take(gu, stage, at_u, at, q);
#pragma unroll
            for (int j = q * UN; j < (q + 1) * UN; ++j) {
                V e[N], hn[N], f[N], y[N];
                above(pz, ph, pd, j, e, hn, f, y);
                if (pre) {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        if (FULL) e[i] = add_(e[i], n0);
                        e[i] = fma_(hn[i], n1, e[i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < N; ++i) f[i] = mul_(e[i], res);
                *reinterpret_cast<Pack<T, U>*>(&px.v[(j % UN) * U]) = narrow<T, U>(f);
                if (gu) {
                    V un[N], k[N];
                    widen(unit(pu, j % UN), un);
                    widen(*at_k(j), k);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        if (post) un[i] = mul_(add_(un[i], neg1), rs1);
                        const V d = mul_(e[i], branch);
                        s1[j][i] = fma_(d, un[i], s1[j][i]);
                        if (FULL) s2[FULL ? j : 0][i] = add_(s2[FULL ? j : 0][i], d);
                        if (post) {
                            e[i] = fma_(e[i], k[i], FULL ? fma_(un[i], k1, k0) : mul_(un[i], k1));
                            e[i] = mul_(e[i], out1);
                        } else {
                            e[i] = mul_(d, k[i]);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < N; ++i) e[i] = mul_(e[i], branch);
                }
                *reinterpret_cast<Pack<T, U>*>(&pu.v[(j % UN) * U]) = narrow<T, U>(e);
            }
            *reinterpret_cast<P*>(dx + at + q * step) = px;
            if (du) *reinterpret_cast<P*>(du + at + q * step) = pu;
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
                *at_k(j) = *reinterpret_cast<const F*>(s1[j]);
                if (FULL) *at_w2(j) = *reinterpret_cast<const F*>(s2[FULL ? j : 0]);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    s1[j][i] = both<V>(0.f);
                    if (FULL) s2[FULL ? j : 0][i] = both<V>(0.f);
                }
            }
#pragma unroll 1
            for (int j = 0; b.part && j < np * UN; ++j) {
                const F x = *at_k(j), y = FULL ? *at_w2(j) : x;
                F a = *at_sum(0, j), e = FULL ? *at_sum(1, j) : x;
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
                *at_sum(0, j) = a;
                if (FULL) *at_sum(1, j) = e;
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
            widen(*at_sum(0, j), s1[j]);
            if (FULL) widen(*at_sum(1, j), s2[FULL ? j : 0]);
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
                    const V* from = n == 0 ? sp[j] : n == SUMS / 2 ? s1[j] : n == 1 ? sq[FULL ? j : 0] : s2[FULL ? j : 0];
                    F f = *reinterpret_cast<const F*>(from);
                    F* const p = reinterpret_cast<F*>(to + n * s.d + column(j));  // d is a multiple of the unit
                    if (k) {
                        const F old = *p;
#pragma unroll
                        for (int i = 0; i < U; ++i) f.v[i] += old.v[i];
                    }
                    *p = f;
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
    const int tensors = (b.dz ? 2 : 0) + (b.dh ? 1 : 0) + (b.u ? 1 : 0);
    const size_t slot = (size_t)threads * s.pieces * vec * sizeof(T) * tensors;
    const size_t wbytes = (size_t)threads * values * 4 * 2;
    const size_t room = threads > 256 ? RB_SMEM_MOST : RB_SMEM_MOST / 2;  // two CTAs of up to 256 threads a SM
    const bool direct = vec * sizeof(T) < 4 || values == 32;  // 2-byte pieces cannot be fetched asynchronously
    s.slots = direct ? 1 : wbytes + 3 * slot <= room ? 3 : wbytes + 2 * slot <= room ? 2 : 1;
    size_t smem = wbytes + (direct ? 0 : s.slots * slot);
    if (s.groups > 1 && smem < (size_t)(full ? 4 : 2) * s.d * 4) smem = (size_t)(full ? 4 : 2) * s.d * 4;
    auto go = [&](auto width, auto columns, auto whole, auto straight) {
        constexpr auto kernel =
            &rn_backward_kernel<T, decltype(width)::value, decltype(columns)::value, decltype(whole)::value, decltype(straight)::value>;
        const cudaError_t e = allow_smem<kernel>(RB_SMEM_MOST);
        if (e != cudaSuccess) return e;
        return launch_k(kernel, dim3(ctas), dim3(threads), smem, st, true, s, w, b, (int)grouped, (int)wbytes);
    };
    auto kinds = [&](auto width, auto columns, auto straight) {
        return full ? go(width, columns, std::true_type(), straight) : go(width, columns, std::false_type(), straight);
    };
    constexpr int VEC = 16 / sizeof(T);
    if (vec == 1)
        return values == 32 ? kinds(Int<1>(), Int<32>(), std::true_type())
                            : kinds(Int<1>(), Int<16>(), std::integral_constant<bool, (sizeof(T) < 4)>());
    return values == 32 ? kinds(Int<VEC>(), Int<32>(), std::true_type()) : kinds(Int<VEC>(), Int<16>(), std::false_type());
}

}  // namespace moe
