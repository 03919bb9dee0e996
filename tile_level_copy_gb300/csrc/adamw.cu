// AdamW over a list of tensors in one launch, states in 32 or in 8 bits.
//
//   g' = g * grad_scale
//   m  = beta1 m + (1 - beta1) g'            v = beta2 v + (1 - beta2) g'^2
//   p  = p (1 - lr wd) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
//
// Every value is read and written once, so the bound is HBM traffic: 28 bytes a value with fp32
// states, bf16 gradients and a bf16 copy, 16 with 8-bit states. The list travels in the launch's
// parameters (no table in device memory to keep in step with the caller's pointers, nothing to copy
// before the launch). So do the step's numbers: a captured launch is the same step at every replay.
// Measured with 24 tensors, 149 million values, bf16 gradients and copies: fp32 states 623 us, 6.7 TB/s
// (98 % of a copy's rate); 8-bit states 467 us, 5.1 TB/s: decoding, the roots and the random roundings take 73
// instructions a value, which fill 59 % of the issue slots (270 us), in long chains, and a thread loads four fours
// and works through them with no load in flight; reading 8-bit states back 250 us, 6.0 TB/s.
//
// 8-bit states. A block of 128 consecutive values has one power-of-two scale for m and one for v, so
// scaling is exact and costs no precision; within a block m keeps 4 exponent bits and 3 mantissa
// bits beside its sign, v (never negative, and spread over twice the exponent range) 5 and 3. Both
// averages change by less than half a rounding step a call (v by 0.1 % with beta2 = 0.999, against
// steps of 6-12 %), so rounding to nearest would never move them: the rounding is stochastic, up
// with a probability equal to the part that is cut off. A value scaled to its code's exponent
// range is an fp32 number whose top bits are the code (subnormal codes are subnormal fp32 numbers),
// so encoding is: add 20 random bits to the bit pattern, shift right by 20.
#include <cuda_fp16.h>
#include <math.h>

#include "host_internal.h"
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int AW_THREADS = 256;
constexpr int AW_CHUNK = 4096;  // values of a tensor that a CTA takes at a time
constexpr int AW_BLOCK = MOE_ADAMW_BLOCK;
static_assert(AW_CHUNK % AW_BLOCK == 0, "a chunk holds whole blocks");

struct AwTensor {
    void* p;
    const void* g;
    __nv_bfloat16* copy;
    void* m;
    void* v;
    uint8_t* ms;
    uint8_t* vs;
    int64_t n;
    int64_t base;
};

enum : uint8_t { AW_P16 = 1, AW_G16 = 2, AW_VEC = 4 };  // bf16 p, bf16 g, pointers aligned for vectors

template <int MAXT>
struct AwList {
    AwTensor t[MAXT];
    int32_t first[MAXT + 1];  // first chunk of each tensor
    uint8_t flags[MAXT];
    int32_t count;
};

struct AwScalars {
    float b1, b1c, b2, b2c;  // beta1, 1 - beta1, beta2, 1 - beta2
    float decay, step, vscale, eps;
    uint32_t k0, k1;
    int flush;  // eps is large enough for roots of subnormal values to be taken as zero
    const float* grad_scale;
};

__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x, uint32_t k) {
    // multiply-xorshift rounds (the constants of Wellons' published low-bias 32-bit mixer), with a
    // second key added between the two
    x ^= x >> 16;
    x *= 0x7FEB352Du;
    x = (x ^ (x >> 15)) + k;
    x *= 0x846CA68Bu;
    return x ^ (x >> 16);
}

// m and v of one value. The products and sums are rounded one by one (no contraction), so that a
// state in 8 bits, whose rounding turns on every bit, is the one the formulas give in fp32.
__device__ __forceinline__ void moments(const AwScalars& s, float g, float& m, float& v) {
    m = __fadd_rn(__fmul_rn(m, s.b1), __fmul_rn(g, s.b1c));
    v = __fadd_rn(__fmul_rn(v, s.b2), __fmul_rn(__fmul_rn(g, g), s.b2c));
}
__device__ __forceinline__ float updated(const AwScalars& s, float p, float m, float v) {
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return p * s.decay - s.step * __fdividef(m, r * s.vscale + s.eps);
}

struct Four {
    float a[4];
};
template <bool VEC>
__device__ __forceinline__ Four load4_f32(const void* base, int64_t i, int k) {
    const float* p = static_cast<const float*>(base) + i;
    Four r{{0.f, 0.f, 0.f, 0.f}};
    if (VEC && k == 4) {
        const float4 q = *reinterpret_cast<const float4*>(p);
        r.a[0] = q.x, r.a[1] = q.y, r.a[2] = q.z, r.a[3] = q.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < k) r.a[j] = p[j];
    }
    return r;
}
template <bool VEC>
__device__ __forceinline__ Four load4_bf16(const void* base, int64_t i, int k) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(base) + i;
    Four r{{0.f, 0.f, 0.f, 0.f}};
    if (VEC && k == 4) {
        const uint2 q = *reinterpret_cast<const uint2*>(p);
        r.a[0] = __uint_as_float(q.x << 16), r.a[1] = __uint_as_float(q.x & 0xffff0000u);
        r.a[2] = __uint_as_float(q.y << 16), r.a[3] = __uint_as_float(q.y & 0xffff0000u);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < k) r.a[j] = __bfloat162float(p[j]);
    }
    return r;
}
template <bool VEC>
__device__ __forceinline__ void store4_f32(void* base, int64_t i, int k, const Four& r) {
    float* p = static_cast<float*>(base) + i;
    if (VEC && k == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(r.a[0], r.a[1], r.a[2], r.a[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < k) p[j] = r.a[j];
    }
}
template <bool VEC>
__device__ __forceinline__ void store4_bf16(void* base, int64_t i, int k, const Four& r) {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(base) + i;
    if (VEC && k == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(r.a[0], r.a[1]), pack_bf16x2(r.a[2], r.a[3]));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < k) p[j] = __float2bfloat16_rn(r.a[j]);
    }
}
template <bool VEC>
__device__ __forceinline__ uint32_t load4_u8(const void* base, int64_t i, int k) {
    const uint8_t* p = static_cast<const uint8_t*>(base) + i;
    if (VEC && k == 4) return *reinterpret_cast<const uint32_t*>(p);
    uint32_t r = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < k) r |= (uint32_t)p[j] << (8 * j);
    return r;
}
template <bool VEC>
__device__ __forceinline__ void store4_u8(void* base, int64_t i, int k, uint32_t r) {
    uint8_t* p = static_cast<uint8_t*>(base) + i;
    if (VEC && k == 4) {
        *reinterpret_cast<uint32_t*>(p) = r;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < k) p[j] = (uint8_t)(r >> (8 * j));
    }
}

// ---- 8-bit codes -------------------------------------------------------------------------------
constexpr int M_TOP = 7, V_TOP = 15;  // a block's largest value is scaled into [2^TOP, 2^(TOP + 1))

__device__ __forceinline__ float scale_value(uint32_t s) {
    return s == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(s << 23);  // 0: 0
}
__device__ __forceinline__ float m_value(uint32_t c, float scale) {
    const float a = __fmul_rn(__uint_as_float((c & 0x7fu) << 20), 0x1p120f);
    return __fmul_rn(__uint_as_float(__float_as_uint(a) | ((c & 0x80u) << 24)), scale);
}
__device__ __forceinline__ float v_value(uint32_t c, float scale) {
    return __fmul_rn(__fmul_rn(__uint_as_float(c << 20), 0x1p112f), scale);
}
// Scale byte for a block whose largest magnitude has the bit pattern `most`.
__device__ __forceinline__ uint32_t block_scale(uint32_t most, int top) {
    if (most >= 0x7f800000u) return 255u;
    const int k = (int)(most >> 23) - 127 - top;
    return (uint32_t)((k < -126 ? -126 : k) + 127);  // k <= 127 - 7
}
__device__ __forceinline__ float inverse_scale(uint32_t s) {
    return s == 255u ? 0.f : __uint_as_float((254u - s) << 23);
}
// 20 random bits from 16: the half step keeps the rounding centred.
__device__ __forceinline__ uint32_t rnd20(uint32_t r16) { return (r16 << 4) + 8u; }

// One CTA's chunk of one tensor.
template <bool EIGHT, bool VEC>
__device__ __forceinline__ void chunk_step(const AwTensor& t, uint32_t flags, const AwScalars& s, float gs, int64_t at) {
    const int64_t left = t.n - at;
    const int len = left < AW_CHUNK ? (int)left : AW_CHUNK;
    const bool p16 = flags & AW_P16, g16 = flags & AW_G16;
    // a warp takes 128 consecutive values (one block of an 8-bit state), a lane four of them
#pragma unroll 2
    for (int o = threadIdx.x * 4; o < AW_CHUNK; o += AW_THREADS * 4) {
        if ((o & ~(AW_BLOCK - 1)) >= len) break;  // the same for the whole warp
        const int k = min(4, max(0, len - o));
        const int64_t i = at + o;
        Four p = p16 ? load4_bf16<VEC>(t.p, i, k) : load4_f32<VEC>(t.p, i, k);
        Four g = g16 ? load4_bf16<VEC>(t.g, i, k) : load4_f32<VEC>(t.g, i, k);
        Four m, v;
        if (EIGHT) {
            const int64_t b = i / AW_BLOCK;
            const float ms = scale_value(t.ms[b]), vs = scale_value(t.vs[b]);
            const uint32_t mc = load4_u8<VEC>(t.m, i, k), vc = load4_u8<VEC>(t.v, i, k);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                m.a[j] = m_value((mc >> (8 * j)) & 0xffu, ms);
                v.a[j] = v_value((vc >> (8 * j)) & 0xffu, vs);
            }
        } else {
            m = load4_f32<VEC>(t.m, i, k);
            v = load4_f32<VEC>(t.v, i, k);
        }
        uint32_t mm = 0, vm = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            moments(s, __fmul_rn(g.a[j], gs), m.a[j], v.a[j]);
            p.a[j] = updated(s, p.a[j], m.a[j], v.a[j]);
            if (EIGHT && j < k) {
                mm = max(mm, __float_as_uint(m.a[j]) & 0x7fffffffu);
                vm = max(vm, __float_as_uint(v.a[j]) & 0x7fffffffu);
            }
        }
        if (p16) store4_bf16<VEC>(t.p, i, k, p);
        else store4_f32<VEC>(t.p, i, k, p);
        if (t.copy) store4_bf16<VEC>(t.copy, i, k, p);
        if (EIGHT) {
            const uint32_t sm = block_scale(__reduce_max_sync(0xffffffffu, mm), M_TOP);
            const uint32_t sv = block_scale(__reduce_max_sync(0xffffffffu, vm), V_TOP);
            const float im = inverse_scale(sm), iv = inverse_scale(sv);
            const uint64_t idx = (uint64_t)(t.base + i);
            uint32_t mc = 0, vc = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint64_t e = idx + j;
                const uint32_t r = mix32((uint32_t)e ^ s.k0, s.k1 + (uint32_t)(e >> 32) * 0x9E3779B9u);
                const uint32_t mb = __float_as_uint(__fmul_rn(__fmul_rn(m.a[j], im), 0x1p-120f));
                const uint32_t vb = __float_as_uint(__fmul_rn(__fmul_rn(v.a[j], iv), 0x1p-112f));
                const uint32_t cm = (((mb & 0x7fffffffu) + rnd20(r & 0xffffu)) >> 20) | ((mb >> 24) & 0x80u);
                const uint32_t cv = ((vb & 0x7fffffffu) + rnd20(r >> 16)) >> 20;
                mc |= (sm == 255u ? 0u : cm & 0xffu) << (8 * j);
                vc |= (sv == 255u ? 0u : cv & 0xffu) << (8 * j);
            }
            store4_u8<VEC>(t.m, i, k, mc);
            store4_u8<VEC>(t.v, i, k, vc);
            if ((threadIdx.x & 31) == 0) {
                const int64_t b = i / AW_BLOCK;
                t.ms[b] = (uint8_t)sm;
                t.vs[b] = (uint8_t)sv;
            }
        } else {
            store4_f32<VEC>(t.m, i, k, m);
            store4_f32<VEC>(t.v, i, k, v);
        }
    }
}

// ---- whole chunks of aligned tensors ----------------------------------------------------------------
// The same arithmetic two values at a time (f32x2, each operation rounded to nearest, none contracted),
// with the 8-bit form's bit work cut down: with it unvectorised the step took 101 instructions a value and
// 647 us for 149 M values (350 us of memory traffic).
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair2(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 split2(f2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
// Sums of products, one by one: as f32x2 additions they came out contracted with the products (a code in
// 50,000 differed), which __fadd_rn rules out.
__device__ __forceinline__ f2 sum2(f2 a, f2 b) {
    const float2 x = split2(a), y = split2(b);
    return pair2(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float max_abs_nan(float a, float b) {  // the larger magnitude, NaN if either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}

// Four consecutive values: p, g (fp32 or bf16, as bits) and their states' bits.
template <bool EIGHT, bool P16, bool G16>
struct AwFour {
    uint4 p, g, m, v;
    uint32_t ms, vs;
    __device__ __forceinline__ void load(const AwTensor& t, int64_t i) {
        if (P16) {
            const uint2 q = __ldcs(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(t.p) + i));
            p.x = q.x, p.y = q.y;
        } else {
            p = __ldcs(reinterpret_cast<const uint4*>(static_cast<const float*>(t.p) + i));
        }
        if (G16) {
            const uint2 q = __ldcs(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(t.g) + i));
            g.x = q.x, g.y = q.y;
        } else {
            g = __ldcs(reinterpret_cast<const uint4*>(static_cast<const float*>(t.g) + i));
        }
        if (EIGHT) {
            m.x = __ldcs(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.m) + i));
            v.x = __ldcs(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.v) + i));
            ms = t.ms[i / AW_BLOCK];
            vs = t.vs[i / AW_BLOCK];
        } else {
            m = __ldcs(reinterpret_cast<const uint4*>(static_cast<const float*>(t.m) + i));
            v = __ldcs(reinterpret_cast<const uint4*>(static_cast<const float*>(t.v) + i));
        }
    }
    template <bool B16>
    static __device__ __forceinline__ void widen(const uint4& q, f2 (&o)[2]) {
        if (B16) {
            o[0] = pair2(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xffff0000u));
            o[1] = pair2(__uint_as_float(q.y << 16), __uint_as_float(q.y & 0xffff0000u));
        } else {
            o[0] = pair2(__uint_as_float(q.x), __uint_as_float(q.y));
            o[1] = pair2(__uint_as_float(q.z), __uint_as_float(q.w));
        }
    }
    // codes of m: two bytes are two fp8 (e4m3) values
    static __device__ __forceinline__ void widen_m(uint32_t q, uint32_t scale, f2 (&o)[2]) {
        const float f = scale_value(scale);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t w;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(w) : "h"((uint16_t)(q >> (16 * h))));
            const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w));
            o[h] = mul2(pair2(x.x, x.y), pair2(f, f));
        }
    }
    static __device__ __forceinline__ void widen_v(uint32_t q, uint32_t scale, f2 (&o)[2]) {
        // byte j at bits 20-27: an fp32 number that is 2^-112 of the code's
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float a = __uint_as_float(__byte_perm(q, 0, h ? 0x4244 : 0x4044) << 4);
            const float b = __uint_as_float(__byte_perm(q, 0, h ? 0x4344 : 0x4144) << 4);
            const f2 x = pair2(a, b);
            if (scale - 1u < 142u) {  // 2^112 and the scale in one factor
                const float f = __uint_as_float((scale + 112u) << 23);
                o[h] = mul2(x, pair2(f, f));
            } else {
                const float f = scale_value(scale);
                o[h] = mul2(mul2(x, pair2(0x1p112f, 0x1p112f)), pair2(f, f));
            }
        }
    }
    __device__ __forceinline__ void step(const AwTensor& t, const AwScalars& s, float gs, int64_t i) {
        f2 P[2], G[2], M[2], V[2];
        widen<P16>(p, P);
        widen<G16>(g, G);
        if (EIGHT) {
            widen_m(m.x, ms, M);
            widen_v(v.x, vs, V);
        } else {
            widen<false>(m, M);
            widen<false>(v, V);
        }
        const f2 scale = pair2(gs, gs), b1 = pair2(s.b1, s.b1), b1c = pair2(s.b1c, s.b1c), b2 = pair2(s.b2, s.b2);
        const f2 b2c = pair2(s.b2c, s.b2c), vscale = pair2(s.vscale, s.vscale), eps = pair2(s.eps, s.eps);
        const f2 decay = pair2(s.decay, s.decay), back = pair2(-s.step, -s.step);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f2 a = mul2(G[h], scale);
            M[h] = sum2(mul2(M[h], b1), mul2(a, b1c));
            V[h] = sum2(mul2(V[h], b2), mul2(mul2(a, a), b2c));
            const float2 v = split2(V[h]);
            const float2 d = split2(fma2(pair2(root(s, v.x), root(s, v.y)), vscale, eps));
            const f2 u = mul2(M[h], pair2(inverse(s, d.x), inverse(s, d.y)));
            P[h] = fma2(P[h], decay, mul2(u, back));
        }
        const float2 p0 = split2(P[0]), p1 = split2(P[1]);
        const uint2 p16 = make_uint2(pack_bf16x2(p0.x, p0.y), pack_bf16x2(p1.x, p1.y));
        if (P16) __stcs(reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(t.p) + i), p16);
        else __stcs(reinterpret_cast<float4*>(static_cast<float*>(t.p) + i), make_float4(p0.x, p0.y, p1.x, p1.y));
        if (t.copy) __stcs(reinterpret_cast<uint2*>(t.copy + i), p16);
        const float2 m0 = split2(M[0]), m1 = split2(M[1]), v0 = split2(V[0]), v1 = split2(V[1]);
        if (!EIGHT) {
            __stcs(reinterpret_cast<float4*>(static_cast<float*>(t.m) + i), make_float4(m0.x, m0.y, m1.x, m1.y));
            __stcs(reinterpret_cast<float4*>(static_cast<float*>(t.v) + i), make_float4(v0.x, v0.y, v1.x, v1.y));
            return;
        }
        const float mm = max_abs_nan(max_abs_nan(m0.x, m0.y), max_abs_nan(m1.x, m1.y));
        const float vm = max_abs_nan(max_abs_nan(v0.x, v0.y), max_abs_nan(v1.x, v1.y));
        const uint32_t sm = block_scale(__reduce_max_sync(0xffffffffu, __float_as_uint(mm)), M_TOP);
        const uint32_t sv = block_scale(__reduce_max_sync(0xffffffffu, __float_as_uint(vm)), V_TOP);
        uint32_t mb[4], vb[4];
        shifted(M, sm, 7u, 0x1p-120f, mb);
        shifted(V, sv, 15u, 0x1p-112f, vb);
        const uint64_t idx = (uint64_t)(t.base + i);
        const uint32_t lo = (uint32_t)idx, key = s.k1 + (uint32_t)(idx >> 32) * 0x9E3779B9u;
        const uint32_t wrap = lo > 0xfffffffcu ? 0x9E3779B9u : 0u;  // the index's low word overflows within the four
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t e = lo + j;
            const uint32_t r = mix32(e ^ s.k0, wrap && e < lo ? key + wrap : key);
            // code to the top byte: m's 7 bits come from 20-26 and its sign stays, v's 8 from 20-27
            const uint32_t a = mb[j] + ((r << 4) & 0xffff0u) + 8u;
            mb[j] = ((a << 4) & 0x7f000000u) | (a & 0x80000000u);
            vb[j] = (vb[j] + ((r >> 12) & 0xffff0u) + 8u) << 4;
        }
        const uint32_t mc = __byte_perm(__byte_perm(mb[0], mb[1], 0x0073), __byte_perm(mb[2], mb[3], 0x0073), 0x5410);
        const uint32_t vc = __byte_perm(__byte_perm(vb[0], vb[1], 0x0073), __byte_perm(vb[2], vb[3], 0x0073), 0x5410);
        __stcs(reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.m) + i), sm == 255u ? 0u : mc);
        __stcs(reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.v) + i), sv == 255u ? 0u : vc);
        if ((threadIdx.x & 31) == 0) {
            t.ms[i / AW_BLOCK] = (uint8_t)sm;
            t.vs[i / AW_BLOCK] = (uint8_t)sv;
        }
    }
    // Values over their scale, times `down` (2^-(127 - bias)): the bits that encoding starts from. Both
    // factors are one, 2^(bias - scale), where it is a normal number.
    static __device__ __forceinline__ void shifted(const f2 (&x)[2], uint32_t scale, uint32_t bias, float down, uint32_t (&o)[4]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            f2 y;
            if (scale < 127u + bias) {
                const float f = __uint_as_float((127u + bias - scale) << 23);
                y = mul2(x[h], pair2(f, f));
            } else {
                const float f = inverse_scale(scale);
                y = mul2(mul2(x[h], pair2(f, f)), pair2(down, down));
            }
            const float2 z = split2(y);
            o[2 * h] = __float_as_uint(z.x);
            o[2 * h + 1] = __float_as_uint(z.y);
        }
    }
    // Square root and reciprocal to a few units of the last place, subnormals as zero where eps (at least
    // 1e-10, against at most 2^-63 of a subnormal v's root) makes that invisible.
    static __device__ __forceinline__ float root(const AwScalars& s, float v) {
        float r;
        if (s.flush) asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
        else asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
        return r;
    }
    static __device__ __forceinline__ float inverse(const AwScalars& s, float v) {
        float r;
        if (s.flush) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
        else r = __fdividef(1.0f, v);
        return r;
    }
};

template <bool EIGHT, bool P16, bool G16>
__device__ __forceinline__ void chunk_whole(const AwTensor& t, const AwScalars& s, float gs, int64_t at) {
    // fours of a thread in flight: with 8-bit states 4 (467 us; 2: 641, and 707 with one more CTA a SM), with
    // 32-bit states 1 in more CTAs (624 us; 2: 637, 4: 661)
    constexpr int AHEAD = EIGHT ? 4 : 1;
    const int64_t i = at + threadIdx.x * 4;
#pragma unroll 1
    for (int o = 0; o < AW_CHUNK; o += AW_THREADS * 4 * AHEAD) {
        AwFour<EIGHT, P16, G16> f[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) f[k].load(t, i + o + k * AW_THREADS * 4);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) f[k].step(t, s, gs, i + o + k * AW_THREADS * 4);
    }
}

template <int MAXT>
__device__ __forceinline__ int tensor_of(const AwList<MAXT>& l, int c) {
    int lo = 0, hi = l.count - 1;  // the last tensor whose first chunk is at or before c
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (l.first[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

constexpr int AW_CTAS_8 = 3;  // CTAs on a SM, 8-bit states

template <bool EIGHT, int MAXT>
__global__ void __launch_bounds__(AW_THREADS, EIGHT ? AW_CTAS_8 : 5) adamw_kernel(const __grid_constant__ AwList<MAXT> l, const AwScalars s) {
    griddep_wait();
    griddep_launch();
    const float gs = s.grad_scale ? *s.grad_scale : 1.0f;
    for (int c = blockIdx.x; c < l.first[l.count]; c += gridDim.x) {
        const int i = tensor_of(l, c);
        const int64_t at = (int64_t)(c - l.first[i]) * AW_CHUNK;
        const AwTensor t = l.t[i];
        const uint32_t f = l.flags[i];
        if (!(f & AW_VEC)) chunk_step<EIGHT, false>(t, f, s, gs, at);
        else if (t.n - at < AW_CHUNK) chunk_step<EIGHT, true>(t, f, s, gs, at);
        else if (f & AW_P16) (f & AW_G16) ? chunk_whole<EIGHT, true, true>(t, s, gs, at) : chunk_whole<EIGHT, true, false>(t, s, gs, at);
        else (f & AW_G16) ? chunk_whole<EIGHT, false, true>(t, s, gs, at) : chunk_whole<EIGHT, false, false>(t, s, gs, at);
    }
}

// Values of 8-bit states (AwTensor.p: fp32 m, .copy: fp32 v, each may be null).
template <int MAXT>
__global__ void __launch_bounds__(AW_THREADS) adamw_read_kernel(const __grid_constant__ AwList<MAXT> l) {
    griddep_wait();
    griddep_launch();
    for (int c = blockIdx.x; c < l.first[l.count]; c += gridDim.x) {
        const int ti = tensor_of(l, c);
        const AwTensor& t = l.t[ti];
        const int64_t at = (int64_t)(c - l.first[ti]) * AW_CHUNK, left = t.n - at;
        const int len = left < AW_CHUNK ? (int)left : AW_CHUNK;
        const bool vec = l.flags[ti] & AW_VEC;
        if (vec && len == AW_CHUNK && t.p && t.copy) {  // whole chunks: 16 values of a thread in flight
            constexpr int N = AW_CHUNK / (AW_THREADS * 4);
            const int64_t i = at + threadIdx.x * 4;
            uint32_t m[N], v[N];
            float ms[N], vs[N];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int64_t e = i + k * AW_THREADS * 4;
                m[k] = load4_u8<true>(t.m, e, 4);
                v[k] = load4_u8<true>(t.v, e, 4);
                ms[k] = scale_value(t.ms[e / AW_BLOCK]);
                vs[k] = scale_value(t.vs[e / AW_BLOCK]);
            }
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int64_t e = i + k * AW_THREADS * 4;
                Four a, b;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    a.a[j] = m_value((m[k] >> (8 * j)) & 0xffu, ms[k]);
                    b.a[j] = v_value((v[k] >> (8 * j)) & 0xffu, vs[k]);
                }
                store4_f32<true>(t.p, e, 4, a);
                store4_f32<true>(t.copy, e, 4, b);
            }
            continue;
        }
        for (int o = threadIdx.x * 4; o < len; o += AW_THREADS * 4) {
            const int k = min(4, len - o);
            const int64_t i = at + o, b = i / AW_BLOCK;
            if (t.p) {
                const float sc = scale_value(t.ms[b]);
                const uint32_t q = vec ? load4_u8<true>(t.m, i, k) : load4_u8<false>(t.m, i, k);
                Four r;
#pragma unroll
                for (int j = 0; j < 4; ++j) r.a[j] = m_value((q >> (8 * j)) & 0xffu, sc);
                if (vec) store4_f32<true>(t.p, i, k, r);
                else store4_f32<false>(t.p, i, k, r);
            }
            if (t.copy) {
                const float sc = scale_value(t.vs[b]);
                const uint32_t q = vec ? load4_u8<true>(t.v, i, k) : load4_u8<false>(t.v, i, k);
                Four r;
#pragma unroll
                for (int j = 0; j < 4; ++j) r.a[j] = v_value((q >> (8 * j)) & 0xffu, sc);
                if (vec) store4_f32<true>(t.copy, i, k, r);
                else store4_f32<false>(t.copy, i, k, r);
            }
        }
    }
}

// Lists longer than MAXT tensors take several launches; a short list takes the small parameter block.
constexpr int AW_SMALL = 32, AW_LARGE = 352;
static_assert(sizeof(AwList<AW_LARGE>) + sizeof(AwScalars) < 32000, "launch parameters");

// Calls run(list, chunks) for each launch's part of the list, made by put(i, &tensor, &flags).
template <int MAXT, typename Put, typename Run>
int over_list(int count, Put put, Run run) {
    AwList<MAXT> l;
    for (int i = 0; i < count;) {
        int k = 0;
        int64_t chunks = 0;
        for (; i < count && k < MAXT; ++i) {
            uint8_t f = 0;
            put(i, &l.t[k], &f);
            if (l.t[k].n == 0) continue;
            const int64_t more = (l.t[k].n + AW_CHUNK - 1) / AW_CHUNK;
            if (chunks + more > INT_MAX) break;
            l.flags[k] = f;
            l.first[k++] = (int32_t)chunks;
            chunks += more;
        }
        if (k == 0) {
            if (i >= count) break;
            return fail(MOE_ERR_ARG, "tensor %d is too long", i);
        }
        l.first[k] = (int32_t)chunks;
        l.count = k;
        const int rc = run(l, (int)chunks);
        if (rc) return rc;
    }
    return MOE_OK;
}

int check_device(DeviceInfo* di) {
    const int rc = device_info(di);
    if (rc) return rc;
    return di->supported ? MOE_OK : fail(MOE_ERR_DEVICE, "current device is not sm_103 (GB300)");
}

// With 8-bit states as many CTAs as run at a time (467 us; eight a SM, two rounds and a part: 488); the
// other forms take the same time with either.
int grid_of(const DeviceInfo& di, int chunks, int per_sm) { return chunks < di.sms * per_sm ? chunks : di.sms * per_sm; }

template <int MAXT>
int step_list(const moe_adamw_config& c, const moe_adamw_tensor* ts, int count, const AwScalars& s,
              const DeviceInfo& di, cudaStream_t st) {
    const bool eight = c.bits == 8;
    return over_list<MAXT>(
        count,
        [&](int i, AwTensor* t, uint8_t* f) {
            const moe_adamw_tensor& a = ts[i];
            *t = AwTensor{a.p, a.g, static_cast<__nv_bfloat16*>(a.copy), a.m, a.v, a.m_scale, a.v_scale, a.n, a.rng_base};
            const size_t sa = eight ? 4 : 16;
            const bool vec = aligned(a.p, a.p_dtype == MOE_DTYPE_F32 ? 16 : 8) &&
                             aligned(a.g, a.g_dtype == MOE_DTYPE_F32 ? 16 : 8) && aligned(a.copy, 8) &&
                             aligned(a.m, sa) && aligned(a.v, sa);
            *f = (a.p_dtype == MOE_DTYPE_BF16 ? AW_P16 : 0) | (a.g_dtype == MOE_DTYPE_BF16 ? AW_G16 : 0) |
                 (vec ? AW_VEC : 0);
        },
        [&](const AwList<MAXT>& l, int chunks) {
            const dim3 grid(grid_of(di, chunks, eight ? AW_CTAS_8 : 8)), block(AW_THREADS);
            const cudaError_t e = eight ? launch_k(adamw_kernel<true, MAXT>, grid, block, 0, st, true, l, s)
                                        : launch_k(adamw_kernel<false, MAXT>, grid, block, 0, st, true, l, s);
            return e == cudaSuccess ? MOE_OK : cuda_fail(e, "AdamW kernel launch");
        });
}

template <int MAXT>
int read_list(const moe_adamw_tensor* ts, int count, float* const* mo, float* const* vo, const DeviceInfo& di,
              cudaStream_t st) {
    return over_list<MAXT>(
        count,
        [&](int i, AwTensor* t, uint8_t* f) {
            const moe_adamw_tensor& a = ts[i];
            float *m = mo ? mo[i] : nullptr, *v = vo ? vo[i] : nullptr;
            *t = AwTensor{m, nullptr, reinterpret_cast<__nv_bfloat16*>(v), a.m, a.v, a.m_scale, a.v_scale,
                          (m || v) ? a.n : 0, 0};
            *f = (aligned(m, 16) && aligned(v, 16) && aligned(a.m, 4) && aligned(a.v, 4)) ? AW_VEC : 0;
        },
        [&](const AwList<MAXT>& l, int chunks) {
            const cudaError_t e =
                launch_k(adamw_read_kernel<MAXT>, dim3(grid_of(di, chunks, 8)), dim3(AW_THREADS), 0, st, true, l);
            return e == cudaSuccess ? MOE_OK : cuda_fail(e, "AdamW state kernel launch");
        });
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

MOE_API int moe_adamw_step(const moe_adamw_config* c, const moe_adamw_tensor* ts, int32_t count,
                           const float* grad_scale, void* stream) {
    clear_error();
    if (!c) return fail(MOE_ERR_ARG, "config is NULL");
    if (c->bits != 32 && c->bits != 8) return fail(MOE_ERR_ARG, "bits=%d must be 32 or 8", c->bits);
    if (c->step < 1) return fail(MOE_ERR_ARG, "step=%lld must be >= 1", (long long)c->step);
    if (!(c->beta1 >= 0 && c->beta1 < 1) || !(c->beta2 >= 0 && c->beta2 < 1))
        return fail(MOE_ERR_ARG, "beta1=%g and beta2=%g must be in [0, 1)", c->beta1, c->beta2);
    if (!(c->eps >= 0) || !isfinite(c->eps) || !isfinite(c->lr) || !isfinite(c->weight_decay))
        return fail(MOE_ERR_ARG, "eps=%g must be >= 0, eps, lr=%g and weight_decay=%g finite", c->eps, c->lr,
                    c->weight_decay);
    for (int i = 0; i < 3; ++i)
        if (c->reserved[i]) return fail(MOE_ERR_ARG, "reserved fields must be zero");
    if (count < 0) return fail(MOE_ERR_ARG, "count=%d must be >= 0", count);
    if (count && !ts) return fail(MOE_ERR_ARG, "tensors is NULL");
    if (!aligned(grad_scale, 4)) return fail(MOE_ERR_ARG, "grad_scale must be 4-byte aligned");
    const bool eight = c->bits == 8;
    int64_t values = 0;
    for (int i = 0; i < count; ++i) {
        const moe_adamw_tensor& t = ts[i];
        if (t.n < 0) return fail(MOE_ERR_ARG, "tensor %d: n=%lld must be >= 0", i, (long long)t.n);
        if ((t.p_dtype != MOE_DTYPE_F32 && t.p_dtype != MOE_DTYPE_BF16) ||
            (t.g_dtype != MOE_DTYPE_F32 && t.g_dtype != MOE_DTYPE_BF16))
            return fail(MOE_ERR_ARG, "tensor %d: p and g must be fp32 or bf16", i);
        if (t.n == 0) continue;
        values += t.n;
        if (!t.p || !t.g || !t.m || !t.v) return fail(MOE_ERR_ARG, "tensor %d: p, g, m or v is NULL", i);
        if (eight && (!t.m_scale || !t.v_scale)) return fail(MOE_ERR_ARG, "tensor %d: m_scale or v_scale is NULL", i);
        if (!aligned(t.p, t.p_dtype == MOE_DTYPE_F32 ? 4 : 2) || !aligned(t.g, t.g_dtype == MOE_DTYPE_F32 ? 4 : 2) ||
            !aligned(t.copy, 2) || (!eight && (!aligned(t.m, 4) || !aligned(t.v, 4))))
            return fail(MOE_ERR_ARG, "tensor %d: a pointer is not aligned to its type", i);
    }
    if (values == 0) return MOE_OK;
    DeviceInfo di;
    const int rc = check_device(&di);
    if (rc) return rc;
    AwScalars s;
    s.b1 = (float)c->beta1;
    s.b1c = (float)(1.0 - c->beta1);
    s.b2 = (float)c->beta2;
    s.b2c = (float)(1.0 - c->beta2);
    s.decay = (float)(1.0 - c->lr * c->weight_decay);
    s.step = (float)(c->lr / (1.0 - pow(c->beta1, (double)c->step)));
    s.vscale = (float)(1.0 / sqrt(1.0 - pow(c->beta2, (double)c->step)));
    s.eps = (float)c->eps;
    s.flush = c->eps >= 1e-10 && c->eps < 1e30;
    s.k0 = mix32((uint32_t)c->seed ^ (uint32_t)c->step, (uint32_t)(c->seed >> 32));
    s.k1 = mix32(s.k0 ^ 0x9E3779B9u, (uint32_t)((uint64_t)c->step >> 32));
    s.grad_scale = grad_scale;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return count <= AW_SMALL ? step_list<AW_SMALL>(*c, ts, count, s, di, st)
                             : step_list<AW_LARGE>(*c, ts, count, s, di, st);
}

MOE_API int moe_adamw_read_state(const moe_adamw_tensor* ts, int32_t count, float* const* m_out, float* const* v_out,
                                 void* stream) {
    clear_error();
    if (count < 0) return fail(MOE_ERR_ARG, "count=%d must be >= 0", count);
    if (count && !ts) return fail(MOE_ERR_ARG, "tensors is NULL");
    int64_t values = 0;
    for (int i = 0; i < count; ++i) {
        const moe_adamw_tensor& t = ts[i];
        const float *m = m_out ? m_out[i] : nullptr, *v = v_out ? v_out[i] : nullptr;
        if (t.n < 0) return fail(MOE_ERR_ARG, "tensor %d: n=%lld must be >= 0", i, (long long)t.n);
        if (t.n == 0 || (!m && !v)) continue;
        values += t.n;
        if ((m && (!t.m || !t.m_scale)) || (v && (!t.v || !t.v_scale)))
            return fail(MOE_ERR_ARG, "tensor %d: a state pointer is NULL", i);
        if (!aligned(m, 4) || !aligned(v, 4)) return fail(MOE_ERR_ARG, "tensor %d: outputs must be 4-byte aligned", i);
    }
    if (values == 0) return MOE_OK;
    DeviceInfo di;
    const int rc = check_device(&di);
    if (rc) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return count <= AW_SMALL ? read_list<AW_SMALL>(ts, count, m_out, v_out, di, st)
                             : read_list<AW_LARGE>(ts, count, m_out, v_out, di, st);
}

}  // extern "C"
