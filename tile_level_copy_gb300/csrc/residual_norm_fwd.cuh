// Forward pass of the residual norm.
//
//   h = a x + c gate * post(u), z = pre(h); a norm is (v - mean) rstd w + b, with mean 0 for the mean-square kind
//
// The pass reads x and u and writes h and z: HBM bounds it. A group of warps shares a row, which comes through shared
// memory by cp.async while the row before is worked on. h is rounded to its type before the second norm (the value
// the backward pass and every other reader sees) and waits in x's place, or in registers, for the pass that writes z.
// 16384 x 4096 bf16, mean-square norms: 101 us, 5.3 TB/s (78 % of a copy's rate); the warps wait for rows and at the sums'
// barriers. 8192 x 4096 fp32 without a norm behind the block: 89 us (89 %). Rows of odd width, 8001 x 2047 bf16: 45 us
// (43 %), as single values are loaded, checked and stored. 5 rows of 4096: 3 us. (Calls that run one behind the other.)
#pragma once

#include "residual_norm.cuh"

namespace moe {
namespace {

constexpr size_t RF_SMEM_MOST = 224 * 1024;
__host__ __device__ constexpr int rf_ctas(int threads) { return threads > 256 ? 1 : 3; }

// Weights are loaded as values that no store changes (no output may share memory with them): else a piece's loads would wait
// for the stores of the piece before.
// One value: `none` where it is not `there`, by a predicated load.
__device__ __forceinline__ float weight(const float* p, bool there, float none) {
    asm("{\n.reg .pred q;\nsetp.ne.u32 q, %2, 0;\n@q ld.global.nc.f32 %0, [%1];\n}" : "+f"(none) : "l"(p), "r"((uint32_t)there));
    return none;
}
template <typename T>
__device__ __forceinline__ float weight(const T* p, bool there, float none) {
    static_assert(sizeof(T) == 2, "16-bit values");
    T v;
    put(v, none);  // (0 and 1 are values of every type)
    uint16_t bits = *reinterpret_cast<const uint16_t*>(&v);
    asm("{\n.reg .pred q;\nsetp.ne.u32 q, %2, 0;\n@q ld.global.nc.u16 %0, [%1];\n}" : "+h"(bits) : "l"(p), "r"((uint32_t)there));
    return num(*reinterpret_cast<const T*>(&bits));
}

template <typename T, int VEC, int NV, int THREADS, bool WF32, bool LAYER, int MODE>
__global__ void __launch_bounds__(THREADS, rf_ctas(THREADS)) rn_forward_kernel(RnShape s, RnWeights w, RnForward f) {
    typedef RnColumns<T, VEC, NV> C;
    typedef typename C::P P;
    constexpr int NP = C::NP, UN = C::UN;
    constexpr int NEXT = MODE == RN_OWN ? NV * THREADS * (int)sizeof(T) : rn_cover<T>(NV, THREADS);  // from x to u, bytes
    constexpr int SLOT = 2 * NEXT;
    // Pieces beyond the row are left out; of ragged rows, whose pieces are two values, they are zeros: a branch a piece kept
    // the loads apart.
    constexpr bool CUT = MODE == RN_OWN;
    constexpr bool KEEP = MODE == RN_RAGGED;  // whether h stays in registers
    __shared__ __align__(16) float red[2][THREADS / 32];
    extern __shared__ __align__(16) uint8_t rf_smem[];
    griddep_wait();
    griddep_launch();
    const int tpr = s.warps * 32, t = threadIdx.x % tpr, group = threadIdx.x / tpr, lane = threadIdx.x & 31;
    C cols(t, s.d);
    asm volatile("" : "+r"(cols.c0)::"memory");  // no load of the weights moves ahead of the wait above
    const T *const x = static_cast<const T*>(f.x), *const u = static_cast<const T*>(f.u);
    T *const h = static_cast<T*>(f.h), *const z = static_cast<T*>(f.z);
    const int64_t stride = (int64_t)gridDim.x * s.groups;
    uint8_t* const own = rf_smem + (MODE == RN_OWN ? threadIdx.x * sizeof(P) : cover_at<T>(group, tpr, NV));
    // the place of piece q of x (0) or u (1) in the slot at `here`: x's is h's later on
    auto at = [&](uint8_t* here, int tensor, int q) { return reinterpret_cast<P*>(here + tensor * NEXT + q * THREADS * (int)sizeof(P)); };
    auto issue = [&](int64_t r, uint8_t* to) {
        if (r < s.rows) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const T* const rows = n ? u : x;
                if (!rows) continue;
                if (MODE == RN_RAGGED) {
                    cover_row(to + n * NEXT, rows, s.rows * s.d, r * s.d, s.d, t, tpr);
                } else {
                    const T* const from = rows + (r * s.d + cols.c0);
#pragma unroll
                    for (int q = 0; q < NP; ++q)
                        if (q < cols.np) copy_async<sizeof(P)>(at(to, n, q), from + q * C::STEP);
                }
            }
        }
        committed();
    };
    int flip = 0;
    auto row_sum = [&](f2 v) {
        float a = warp_sum(total(v));
        if (s.warps == 1) return a;
        // [half][8 warps' sums]: the halves in turn, so one barrier a sum is enough
        float* const r = red[flip] + group * s.warps;
        flip ^= 1;
        if (lane == 0) r[t >> 5] = a;
        named_bar_sync(1 + group, tpr);
        a = lane < s.warps ? r[lane] : 0.f;
        return warp_sum(a);
    };
    // adds the squares of a piece's values, less the mean where there is one, over the columns of the row
    auto squares = [&](const P& p, bool centred, f2 neg, int q, f2 (&sq)[2]) {
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            f2 v = unit_of(p, i);
            if (centred) {
                v = add_(v, neg);
                if (VEC == 1) {  // a value beyond the row is no value
                    const float2 e = split(v);
                    v = pair(cols.inside(q, 0) ? e.x : 0.f, cols.inside(q, 1) ? e.y : 0.f);
                }
            }
            sq[i & 1] = fma_(v, v, sq[i & 1]);
        }
    };
    // vector p of the weights from the row's column on: unit i of piece q; `none` where p is null, 0 beyond the row (where a
    // layer norm takes its mean off as well). Predicated loads: a branch a vector and piece kept them apart.
    auto coefficients = [&](const void* p, float none, int64_t base, int q, f2 (&k)[UN]) {
        base += cols.c0 + q * C::STEP;
        if constexpr (VEC == 1) {
            float a[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool in = cols.inside(q, i);
                if constexpr (WF32) a[i] = weight(static_cast<const float*>(p) + base + 32 * i, in && p, in ? none : 0.f);
                else a[i] = weight(static_cast<const T*>(p) + base + 32 * i, in && p, in ? none : 0.f);
            }
            k[0] = pair(a[0], a[1]);
        } else if constexpr (WF32) {
            const float4* const v = reinterpret_cast<const float4*>(static_cast<const float*>(p) + base);
#pragma unroll
            for (int i = 0; i < VEC / 4; ++i) {
                const float4 e = p ? __ldg(v + i) : make_float4(none, none, none, none);
                k[2 * i] = pair(e.x, e.y);
                k[2 * i + 1] = pair(e.z, e.w);
            }
        } else {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (p) v = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p) + base));
            const P e = *reinterpret_cast<const P*>(&v);
#pragma unroll
            for (int i = 0; i < UN; ++i) k[i] = p ? unit_of(e, i) : both<f2>(none);
        }
    };

    uint8_t* here = own;
    int64_t r = (int64_t)blockIdx.x * s.groups + group;
    for (int k = 0; k < s.slots - 1; ++k) issue(r + k * stride, own + k * SLOT);
    const f2 zero = both<f2>(0.f);
#pragma unroll 1
    for (; r < s.rows; r += stride) {
        if (MODE == RN_RAGGED) {  // the row is there for all its threads, and they are done with the one before
            fetched(s.slots > 1 ? s.slots - 2 : 0);
            named_bar_sync(1 + group, tpr);
        }
        issue(r + (s.slots - 1) * stride, here == own ? own + (s.slots - 1) * SLOT : here - SLOT);
        if (MODE == RN_RAGGED && s.slots == 1) {
            fetched(0);
            named_bar_sync(1 + group, tpr);
        }
        if (MODE == RN_OWN) fetched(s.slots - 1);
        const int64_t row = r * s.d + cols.c0;
        T* const rx = reinterpret_cast<T*>(here + (MODE == RN_RAGGED ? offset_of(x + r * s.d) : 0)) + (MODE == RN_RAGGED ? cols.c0 : 0);
        const T* const ru = reinterpret_cast<const T*>(here + NEXT + (MODE == RN_RAGGED ? offset_of(u + r * s.d) : 0)) + (MODE == RN_RAGGED ? cols.c0 : 0);
        auto take = [&](int n, int q) {  // piece q of x (h) or u
            if (MODE == RN_OWN) return *at(here, n, q);
            return cols.load(n ? ru : rx, q);
        };
        float mu = 0.f, rs = 1.f;
        if (s.post) {
            f2 sq[2] = {zero, zero};
            if (LAYER && s.post == MOE_NORM_LAYER) {
#pragma unroll
                for (int q = 0; q < NP; ++q) {
                    if (CUT && q >= cols.np) break;
                    const P p = take(1, q);
#pragma unroll
                    for (int i = 0; i < UN; ++i) sq[i & 1] = add_(sq[i & 1], unit_of(p, i));
                }
                mu = row_sum(add_(sq[0], sq[1])) * s.inv_d;
                sq[0] = sq[1] = zero;
            }
            const f2 neg = both<f2>(-mu);
            auto over = [&](auto centred) {
#pragma unroll
                for (int q = 0; q < NP; ++q) {
                    if (CUT && q >= cols.np) break;
                    squares(take(1, q), decltype(centred)::value, neg, q, sq);
                }
            };
            if (LAYER && s.post == MOE_NORM_LAYER) over(std::true_type());
            else over(std::false_type());
            rs = rsqrtf(fmaf(row_sum(add_(sq[0], sq[1])), s.inv_d, s.eps));
            if (t == 0 && f.post_stats) f.post_stats[r] = make_float2(mu, rs);
        }
        const f2 a = both<f2>(rs), b = both<f2>(-mu * rs), res = both<f2>(s.res), branch = both<f2>(s.branch);
        const int64_t gate_at = s.gate_rows ? (s.gate_rows >= s.rows ? 0 : r / s.gate_rows * s.d) : 0;
        f2 sum[2] = {zero, zero};  // of h, or of its squares
        P kept[KEEP ? NP : 1];
        auto residual = [&](auto branched) {
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                if (CUT && q >= cols.np) break;
                P px = take(0, q);
                if (decltype(branched)::value) {
                    const P pu = take(1, q);
                    f2 v[UN], k[UN];
#pragma unroll
                    for (int i = 0; i < UN; ++i) v[i] = LAYER ? fma_(unit_of(pu, i), a, b) : mul_(unit_of(pu, i), a);
                    coefficients(w.post_w, 1.f, 0, q, k);
#pragma unroll
                    for (int i = 0; i < UN; ++i) v[i] = mul_(v[i], k[i]);
                    if (LAYER) {
                        coefficients(w.post_b, 0.f, 0, q, k);
#pragma unroll
                        for (int i = 0; i < UN; ++i) v[i] = add_(v[i], k[i]);
                    }
                    coefficients(w.gate, 1.f, gate_at, q, k);
#pragma unroll
                    for (int i = 0; i < UN; ++i) v[i] = mul_(v[i], k[i]);
#pragma unroll
                    for (int i = 0; i < UN; ++i) put_unit(px, i, fma_(v[i], branch, mul_(unit_of(px, i), res)));
                } else {
#pragma unroll
                    for (int i = 0; i < UN; ++i) put_unit(px, i, mul_(unit_of(px, i), res));
                }
                if (h) cols.store(h + row, q, px);
                if (KEEP) kept[KEEP ? q : 0] = px;
                else *at(here, 0, q) = px;
                if (LAYER && s.pre == MOE_NORM_LAYER) {
#pragma unroll
                    for (int i = 0; i < UN; ++i) sum[i & 1] = add_(sum[i & 1], unit_of(px, i));
                } else {
                    squares(px, false, zero, q, sum);
                }
            }
        };
        if (u) residual(std::true_type());
        else residual(std::false_type());
        if (s.pre) {
            mu = 0.f;
            if (LAYER && s.pre == MOE_NORM_LAYER) {
                mu = row_sum(add_(sum[0], sum[1])) * s.inv_d;
                sum[0] = sum[1] = zero;
                const f2 neg = both<f2>(-mu);
#pragma unroll
                for (int q = 0; q < NP; ++q) {
                    if (CUT && q >= cols.np) break;
                    squares(KEEP ? kept[KEEP ? q : 0] : take(0, q), true, neg, q, sum);
                }
            }
            rs = rsqrtf(fmaf(row_sum(add_(sum[0], sum[1])), s.inv_d, s.eps));
            if (t == 0 && f.pre_stats) f.pre_stats[r] = make_float2(mu, rs);
            const f2 a2 = both<f2>(rs), b2 = both<f2>(-mu * rs);
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                if (CUT && q >= cols.np) break;
                P p = KEEP ? kept[KEEP ? q : 0] : take(0, q);
                f2 v[UN], k[UN];
#pragma unroll
                for (int i = 0; i < UN; ++i) v[i] = LAYER ? fma_(unit_of(p, i), a2, b2) : mul_(unit_of(p, i), a2);
                coefficients(w.pre_w, 1.f, 0, q, k);
#pragma unroll
                for (int i = 0; i < UN; ++i) v[i] = mul_(v[i], k[i]);
                if (LAYER) {
                    coefficients(w.pre_b, 0.f, 0, q, k);
#pragma unroll
                    for (int i = 0; i < UN; ++i) v[i] = add_(v[i], k[i]);
                }
#pragma unroll
                for (int i = 0; i < UN; ++i) put_unit(p, i, v[i]);
                cols.store(z + row, q, p);
            }
        }
        here = here == own + (s.slots - 1) * SLOT ? own : here + SLOT;
    }
    fetched(0);
}

}  // namespace

template <typename T>
cudaError_t launch_residual_forward(RnShape s, const RnWeights& w, const RnForward& f, int vec, int sms, cudaStream_t st) {
    // 64 bytes of a row a thread where the rows fill the device; 16 where they would leave it empty (a row then has four
    // times as many warps, and is done sooner)
    constexpr int MANY = 64 / (int)sizeof(T), FEW = 16 / (int)sizeof(T);
    const bool few = s.rows * rn_warps(s.d, MANY) < 16 * sms && rn_warps(s.d, FEW) <= 32;
    // ragged rows of half a warp's values or less: all places of a thread cost their instructions there
    // (40001 x 301 bf16: 64 us instead of 87)
    const bool ragged = vec == 1 || !w.whole, small = few || (ragged && s.d <= 16 * MANY);
    s.warps = rn_warps(s.d, small ? FEW : MANY);
    s.groups = s.warps < 8 && !few ? 8 / s.warps : 1;
    const int threads = 32 * s.warps * s.groups;
    const int64_t n = (s.rows + s.groups - 1) / s.groups;
    auto go = [&](auto width, auto values, auto most, auto wide, auto layer, auto how) {
        constexpr int VEC = decltype(width)::value, NV = decltype(values)::value, THREADS = decltype(most)::value;
        constexpr int MODE = decltype(how)::value;
        constexpr auto kernel = &rn_forward_kernel<T, VEC, NV, THREADS, decltype(wide)::value, decltype(layer)::value, MODE>;
        constexpr size_t slot = 2 * (MODE == RN_OWN ? (size_t)NV * THREADS * sizeof(T) : (size_t)rn_cover<T>(NV, THREADS));
        constexpr size_t room = RF_SMEM_MOST / rf_ctas(THREADS);
        s.slots = 3 * slot <= room ? 3 : 2 * slot <= room ? 2 : 1;
        const int64_t ctas = (int64_t)sms * rf_ctas(THREADS);
        if (n <= ctas) s.slots = 1;  // a row for each group: nothing to fetch ahead
        const cudaError_t e = allow_smem<kernel>(RF_SMEM_MOST);
        if (e != cudaSuccess) return e;
        return launch_k(kernel, dim3((unsigned)(n < ctas ? n : ctas)), dim3(threads), s.slots * slot, st, true, s, w, f);
    };
    auto shaped = [&](auto width, auto wide, auto layer, auto how) {
        if (small) return threads <= 256 ? go(width, Int<FEW>(), Int<256>(), wide, layer, how) : go(width, Int<FEW>(), Int<1024>(), wide, layer, how);
        return threads <= 256 ? go(width, Int<MANY>(), Int<256>(), wide, layer, how) : go(width, Int<MANY>(), Int<1024>(), wide, layer, how);
    };
    auto kinds = [&](auto width, auto wide, auto how) {
        return s.post == MOE_NORM_LAYER || s.pre == MOE_NORM_LAYER ? shaped(width, wide, std::true_type(), how)
                                                                   : shaped(width, wide, std::false_type(), how);
    };
    auto typed = [&](auto width, auto how) {
        if constexpr (sizeof(T) == 4) return kinds(width, std::true_type(), how);
        else return w.f32 ? kinds(width, std::true_type(), how) : kinds(width, std::false_type(), how);
    };
    return ragged ? typed(Int<1>(), Int<RN_RAGGED>()) : typed(Int<16 / sizeof(T)>(), Int<RN_OWN>());
}

}  // namespace moe
