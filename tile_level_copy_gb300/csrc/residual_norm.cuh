// Shapes, columns and values that the passes of the residual norm share.
#pragma once

#include "row_values.cuh"

namespace moe {

constexpr int RN_MAX_D = 16384;

// How a launch's threads share the rows: groups of `warps` warps, `groups` of them in a CTA, with `slots` rows of each
// group in shared memory.
struct RnShape {
    int64_t rows, gate_rows;  // gate_rows 0: no gate
    int64_t chunk;            // backward: consecutive rows of a group of warps
    int d, warps, groups, slots;
    int post, pre;            // MOE_NORM_*
    float eps, inv_d, res, branch;
};
struct RnWeights {
    const void *post_w, *post_b, *gate, *pre_w, *pre_b;
    bool f32;    // fp32, or the rows' type
    bool whole;  // every vector that is there is aligned for whole pieces
};
struct RnForward {
    const void *x, *u;
    void *h, *z;
    float2 *post_stats, *pre_stats;
};
struct RnBackward {
    const void *dz, *dh, *u, *h;
    const float2 *post_stats, *pre_stats;
    void *dx, *du;
    float* part;   // the CTAs' sums
    float* gpart;  // [groups of warps][2][d]: sums of the gates whose rows lie in more than one group of warps
    float* gsum;   // [groups of warps][2][d], with more than one gate: sums of post_w's and post_b's gradients so far
    void* dgate;
};

// Launch the passes on rows of T (files of their own for each type); vec: values of a 16-byte piece, or 1.
template <typename T>
cudaError_t launch_residual_forward(RnShape s, const RnWeights& w, const RnForward& f, int vec, int sms, cudaStream_t st);
template <typename T>
cudaError_t launch_residual_backward(RnShape s, const RnWeights& w, const RnBackward& b, int vec, bool full, bool grouped,
                                     int ctas, cudaStream_t st);

inline int rn_warps(int d, int values) { return (d + 32 * values - 1) / (32 * values); }
// Backward: values of a thread. With layer norms short rows take 8 where the rows are fp32 (8192 x 2048: 74 us instead of 80)
// or groups of them have gates (a gate a row, 16384 x 2048 bf16: 425 us instead of 514), else 16 (16384 x 2048 bf16: 92 us
// instead of 98); 32 of them spill, and only rows above 8192 need them.
inline int rn_backward_values(int d, int dtype, bool full, bool grouped) {
    return full && (grouped || dtype == MOE_DTYPE_F32) && d <= 2048 ? 8 : d <= 8192 ? 16 : 32;
}

namespace {

// How rows reach their readers. RN_OWN: a thread fetches the pieces that it reads itself, so no barrier guards the slots.
// RN_RAGGED: rows of odd addresses, whose values only loads of one value could fetch: the threads of a row fetch the
// 16-byte pieces that cover it and read single values from them, one barrier a row. RN_DIRECT: values are read from
// global memory wherever they are needed (rows too wide for a slot).
enum RnMode : int { RN_OWN, RN_RAGGED, RN_DIRECT };

// The columns of a thread, in units of two: a warp has 32 NV neighbouring ones, so that a thread's lie at fixed distances.
// VEC > 1: pieces of VEC neighbouring values, piece q at 32 VEC q. VEC = 1: a unit is two values 32 apart (single
// values of neighbouring threads lie beside one another), a piece is a unit.
template <typename T, int VEC_, int NV>
struct RnColumns {
    static constexpr int VEC = VEC_, PV = VEC == 1 ? 2 : VEC, NP = NV / PV, UN = PV / 2, NU = NV / 2, STEP = VEC == 1 ? 64 : 32 * VEC;
    typedef Pack<T, PV> P;
    int c0, d, np, nv;  // the first column, values of the row, this thread's pieces, its values (VEC = 1)
    __device__ __forceinline__ RnColumns(int t, int d) : d(d) {
        c0 = (t >> 5) * (32 * NV) + (t & 31) * VEC;
        np = c0 < d ? min(NP, (d - c0 + STEP - 1) / STEP) : 0;
        nv = c0 < d ? min(NV, (d - c0 + 31) / 32) : 0;
    }
    __device__ __forceinline__ int column(int j, int i) const {  // of value i of unit j
        return VEC == 1 ? c0 + j * STEP + i * 32 : c0 + (j / UN) * STEP + (j % UN) * 2 + i;
    }
    __device__ __forceinline__ bool inside(int j, int i) const { return VEC == 1 ? 2 * j + i < nv : j / UN < np; }
    // piece q of a row, whose values from column c0 on lie at p (global memory, or its bytes in a slot); values
    // beyond the row are zero
    __device__ __forceinline__ P load(const T* p, int q) const {
        P r;
        if constexpr (VEC == 1) {
            put(r.v[0], 0.f);
            put(r.v[1], 0.f);
            if (inside(q, 0)) r.v[0] = p[q * STEP];
            if (inside(q, 1)) r.v[1] = p[q * STEP + 32];
        } else {
            if (q < np) r = *reinterpret_cast<const P*>(p + q * STEP);
            else memset(&r, 0, sizeof(r));
        }
        return r;
    }
    // the same from a slot of ragged rows, which holds zeros behind the row
    __device__ __forceinline__ P load_padded(const T* p, int q) const {
        P r;
        r.v[0] = p[q * STEP];
        r.v[1] = p[q * STEP + 32];
        return r;
    }
    __device__ __forceinline__ void store(T* p, int q, const P& r) const {
        if constexpr (VEC == 1) {
            if (inside(q, 0)) p[q * STEP] = r.v[0];
            if (inside(q, 1)) p[q * STEP + 32] = r.v[1];
        } else {
            if (q < np) *reinterpret_cast<P*>(p + q * STEP) = r;
        }
    }
};

// Unit j of a piece as fp32; and back. (By words: pieces of two 16-bit values that are copied one by one cost a byte
// permutation each, a quarter of the backward kernel's instructions.)
template <typename T, int VEC>
__device__ __forceinline__ f2 unit_of(const Pack<T, VEC>& p, int j) {
    if constexpr (sizeof(T) == 4) {
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
__device__ __forceinline__ void put_unit(Pack<T, VEC>& p, int j, f2 v) {
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

template <typename T>
__device__ __forceinline__ float value_at(const void* p, bool f32, int64_t i, float none) {
    return !p ? none : f32 ? static_cast<const float*>(p)[i] : num(static_cast<const T*>(p)[i]);
}

// ---- ragged rows
// Bytes of a tensor in a slot: the rows of up to eight groups, each with what covers its ends.
template <typename T>
__host__ __device__ constexpr int rn_cover(int values, int threads) { return values * threads * (int)sizeof(T) + 8 * 32; }
// Where a group's rows start in it.
template <typename T>
__device__ __forceinline__ int cover_at(int group, int tpr, int values) { return group * (tpr * values * (int)sizeof(T) + 32); }
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
    if (start >= lo && start + 16 * pieces <= hi) {
        for (int i = t; i < pieces; i += threads) copy_async<16>(to + 16 * i, start + 16 * i);
        return;
    }
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

// Zeros behind a row in its slot, up to the end of the pieces that a row may take, by the lanes of the warp that fetched the
// row's last piece (its number modulo the row's threads tells which did), once it is there for all of them. A row's last piece is
// last_piece or one more. (What lies behind those that a row may take is zeroed once.)
template <typename T>
__device__ __forceinline__ int last_piece(int d) { return (d * (int)sizeof(T) + 15) / 16 - 1; }
template <typename T>
__device__ __forceinline__ void pad_row(uint8_t* to, const T* rows, int64_t at, int d, bool owner, bool next_owner, int lane) {
    constexpr int size = (int)sizeof(T);
    const int end = offset_of(rows + at) + d * size, most = (16 - size + d * size + 15) / 16 * 16;
    const int b = end + lane * size;  // (fewer than 32 bytes)
    if (((end + 15) / 16 - 1 == last_piece<T>(d) ? owner : next_owner) && b < most) put(*reinterpret_cast<T*>(to + b), 0.f);
}

__device__ __forceinline__ void fetched(int pending) {  // all but the last `pending` groups are there
    if (pending == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (pending == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 2;" ::: "memory");
}

}  // namespace
}  // namespace moe
