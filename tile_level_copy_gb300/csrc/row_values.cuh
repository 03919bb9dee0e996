// Values of rows as they lie in memory and as fp32, sums over warps, and the checks that the row kernels share.
// Sums and products go two at a time (f32x2).
#pragma once

#include "host_internal.h"
#include "moe_internal.cuh"

#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

namespace moe {
namespace {

template <int N>
struct Int {
    static constexpr int value = N;
};

// ---- values, one (float) or two (f2: a pair of fp32 in 64 bits) at a time -------------------------
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 split(f2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 add_(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 mul_(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma_(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float add_(float a, float b) { return a + b; }
__device__ __forceinline__ float mul_(float a, float b) { return a * b; }
__device__ __forceinline__ float fma_(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float total(f2 v) {
    const float2 s = split(v);
    return s.x + s.y;
}
__device__ __forceinline__ float total(float v) { return v; }
template <typename V>
__device__ __forceinline__ V both(float v);
template <>
__device__ __forceinline__ f2 both<f2>(float v) { return pair(v, v); }
template <>
__device__ __forceinline__ float both<float>(float v) { return v; }

// VEC consecutive values of a row as they lie in memory, and as fp32.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
};
template <int VEC>
struct Lanes {
    typedef f2 V;
    static constexpr int N = VEC / 2;
};
template <>
struct Lanes<1> {
    typedef float V;
    static constexpr int N = 1;
};

__device__ __forceinline__ float num(float v) { return v; }
__device__ __forceinline__ float num(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float num(__half v) { return __half2float(v); }
__device__ __forceinline__ void put(float& o, float v) { o = v; }
__device__ __forceinline__ void put(__nv_bfloat16& o, float v) { o = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half& o, float v) { o = __float2half_rn(v); }

template <typename T, int VEC>
__device__ __forceinline__ void widen(const Pack<T, VEC>& p, f2 (&o)[VEC / 2]) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) o[i] = pair(num(p.v[2 * i]), num(p.v[2 * i + 1]));
}
template <int VEC>
__device__ __forceinline__ void widen(const Pack<__nv_bfloat16, VEC>& p, f2 (&o)[VEC / 2]) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&p);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) o[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ void widen(const Pack<T, 1>& p, float (&o)[1]) {
    o[0] = num(p.v[0]);
}
template <typename T, int VEC>
__device__ __forceinline__ std::enable_if_t<(sizeof(T) == 4), Pack<T, VEC>> narrow(const f2 (&f)[VEC / 2]) {
    Pack<T, VEC> r;
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
        const float2 s = split(f[i]);
        put(r.v[2 * i], s.x);
        put(r.v[2 * i + 1], s.y);
    }
    return r;
}
template <typename T, int VEC>
__device__ __forceinline__ std::enable_if_t<(sizeof(T) == 2), Pack<T, VEC>> narrow(const f2 (&f)[VEC / 2]) {
    Pack<T, VEC> r;
    uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
        const float2 s = split(f[i]);
        if constexpr (std::is_same_v<T, __half>) {
            const __half2 h = __floats2half2_rn(s.x, s.y);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            w[i] = pack_bf16x2(s.x, s.y);
        }
    }
    return r;
}
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, 1> narrow(const float (&f)[1]) {
    Pack<T, 1> r;
    put(r.v[0], f[0]);
    return r;
}
// Keeps the compiler from holding a piece's fp32 form from one pass over the row to the next (it would
// take two registers a 16-bit pair and spill): each pass widens it again, one operation a value.
template <typename T, int VEC>
__device__ __forceinline__ void opaque(Pack<T, VEC>& p) {
    if constexpr (sizeof(p) == 2) {
        asm volatile("" : "+h"(*reinterpret_cast<uint16_t*>(&p)));
    } else {
#pragma unroll
        for (int i = 0; i < (int)sizeof(p) / 4; ++i) asm volatile("" : "+r"(reinterpret_cast<uint32_t*>(&p)[i]));
    }
}
// How a launch reads its weights: fp32 or the rows' type, both vectors there and aligned for whole
// pieces, or one value at a time (a null vector stands for `none`).
enum LnWeights : int { LN_W_F32, LN_W_SAME, LN_W_ANY };

template <typename T, int VEC, int W>
__device__ __forceinline__ void weights(const void* w, bool f32, float none, int c,
                                        typename Lanes<VEC>::V (&o)[Lanes<VEC>::N]) {
    if (W == LN_W_SAME) {
        widen(*reinterpret_cast<const Pack<T, VEC>*>(static_cast<const T*>(w) + c), o);
        return;
    }
    const float* p = static_cast<const float*>(w) + c;
    Pack<float, VEC> v;
    if (W == LN_W_F32) {
        constexpr int L = VEC < 4 ? VEC : 4;
#pragma unroll
        for (int i = 0; i < VEC / L; ++i)
            *reinterpret_cast<Pack<float, L>*>(&v.v[L * i]) = *reinterpret_cast<const Pack<float, L>*>(p + L * i);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v.v[i] = !w ? none : f32 ? p[i] : num(static_cast<const T*>(w)[c + i]);
    }
    widen(v, o);
}

__device__ __forceinline__ float warp_sum(float a) {
#pragma unroll
    for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    return a;
}

template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
    else if constexpr (BYTES >= 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(to)), "l"(from), "n"(BYTES) : "memory");
}

__device__ __forceinline__ void committed() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Sums of K values (a power of two up to 32) over a warp: lane l gets the total of value l / (32 / K).
template <int K>
__device__ __forceinline__ float warp_sums(float (&v)[K], int lane) {
#pragma unroll
    for (int half = K / 2, o = 16; half >= 1; half >>= 1, o >>= 1) {
        const bool hi = lane & o;  // this half of the warp keeps the upper half of the values
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float send = hi ? v[i] : v[i + half], keep = hi ? v[i + half] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    float a = v[0];
#pragma unroll
    for (int o = 16 / K; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    return a;
}

size_t dtype_size(int t) { return t == MOE_DTYPE_F32 ? 4 : 2; }

int check_device(DeviceInfo* di) {
    const int rc = device_info(di);
    if (rc) return rc;
    return di->supported ? MOE_OK : fail(MOE_ERR_DEVICE, "current device is not sm_103 (GB300)");
}

// Once per device and kernel: it may take the most shared memory that a launch of it asks for. (What a kernel may
// take is the process's: set to what one call needs, it could be too little for another thread's launch.)
template <auto Kernel>
cudaError_t allow_smem(size_t most) {
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(Kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e == cudaSuccess) done[dev].store(true, std::memory_order_relaxed);
    return e;
}

}  // namespace
}  // namespace moe
