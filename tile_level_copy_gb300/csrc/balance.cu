// Balance loss and z loss of a router with the experts' loads, and the gradient of its logits.
//
//   p = softmax(l), lse = log sum exp(l); of sequence s: n tokens, c[e] pairs, ps[e] = sum of p
//   balance = mean over sequences with n > 0 of E / (k n^2) sum_e c[e] ps[e],  z = mean over tokens of lse^2
//   dl = dloss p (w_b / S' (a - sum_e p a) + 2 w_z / N lse) + the gates' part,  a[e] = E / (k n^2) c[e]
//
// The logits are read once in each direction and dlogits written once: HBM traffic bounds both passes. A row lies in
// the registers of as many lanes as hold it with eight values a lane, so a warp works on 1 to 32 tokens at once.
// Forward: a CTA takes consecutive tokens and keeps its sums of p in registers until the sequence ends; counts
// are integers in shared memory. What it has of a sequence goes to a row of the workspace: CTA and sequence both
// grow along the tokens, so the pair's rank is their sum. A second launch adds the rows up in the order of the
// CTAs (no sum depends on which CTA was first) and its last CTA makes the losses.
#include <math.h>

#include "row_values.cuh"

namespace moe {
namespace {

constexpr int BL_THREADS = 1024, BL_WARPS = BL_THREADS / 32;       // forward: one CTA a SM, so few rows of sums
constexpr int BL_BACK_THREADS = 256, BL_BACK_WARPS = BL_BACK_THREADS / 32, BL_BACK_CTAS = 4;
constexpr int BL_NV = 8;           // logits of a lane
constexpr int BL_MAX_CTAS = 256;   // of the forward pass
constexpr int BL_MAX_E = 256, BL_MAX_K = 8;
constexpr int BL_END_WARPS = 32;   // of the second launch's CTAs, at most

struct BlShape {
    int T, E, k, S, chunk, ctas;  // a CTA takes `chunk` consecutive tokens
    const int32_t* offsets;
    const uint8_t* mask;
};
// Where sequence s starts (s = S: where the last one ends), within [0, T] whatever the caller's array holds.
__device__ __forceinline__ int start_of(const BlShape& s, int i) {
    if (!s.offsets) return i == 0 ? 0 : s.T;
    return min(max(s.offsets[i], 0), s.T);
}
// The sequence of token t: -1 before the first, S behind the last.
__device__ __forceinline__ int sequence_of(const BlShape& s, int t) {
    if (t < start_of(s, 0)) return -1;
    int lo = 0, hi = s.S;  // the last one that starts at or before t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start_of(s, mid) <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Column of a lane's value i: four neighbours (float4 loads) or every LPT-th.
template <int LPT, bool VEC>
__device__ __forceinline__ int column(int lig, int i) {
    return VEC ? ((i >> 2) * LPT + lig) * 4 + (i & 3) : i * LPT + lig;
}
// A lane's values of a row; -inf where there is none.
template <int LPT, bool VEC>
__device__ __forceinline__ void load_row(const float* row, bool there, int E, int lig, float (&x)[BL_NV]) {
    if (VEC) {
#pragma unroll
        for (int q = 0; q < BL_NV / 4; ++q) {
            const int c = (q * LPT + lig) * 4;
            float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (there && c < E) v = *reinterpret_cast<const float4*>(row + c);
            x[4 * q] = v.x, x[4 * q + 1] = v.y, x[4 * q + 2] = v.z, x[4 * q + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < BL_NV; ++i) {
            const int c = i * LPT + lig;
            x[i] = there && c < E ? row[c] : -INFINITY;
        }
    }
}
template <int LPT>
__device__ __forceinline__ float group_sum(float a) {
#pragma unroll
    for (int o = LPT / 2; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    return a;
}
// Sums of two values over a token's lanes, side by side: one lane's half of the group takes each.
template <int LPT>
__device__ __forceinline__ void group_sums(float& a, float& b, int lane) {
    if (LPT == 1) return;
    const bool hi = lane & (LPT / 2);
    const float send = hi ? a : b;
    float v = (hi ? b : a) + __shfl_xor_sync(0xffffffffu, send, LPT / 2);
#pragma unroll
    for (int o = LPT / 4; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const float w = __shfl_xor_sync(0xffffffffu, v, LPT / 2);
    a = hi ? w : v;
    b = hi ? v : w;
}
__device__ __forceinline__ float exponential(float v) {  // (below 2^-126: zero)
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v * 1.4426950408889634f));
    return r;
}
// x becomes exp(x - max); returns the maximum (0 if every value is -inf). The difference is taken first: with logits at
// the type's lowest value the product with log2(e) would overflow.
template <int LPT>
__device__ __forceinline__ float exponentials(float (&x)[BL_NV]) {
    float m = x[0];
#pragma unroll
    for (int i = 1; i < BL_NV; ++i) m = fmaxf(m, x[i]);
#pragma unroll
    for (int o = LPT / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m == -INFINITY) m = 0.f;
#pragma unroll
    for (int i = 0; i < BL_NV; ++i) x[i] = exponential(x[i] - m);
    return m;
}
__device__ __forceinline__ float sum_of(const float (&x)[BL_NV]) {
    float a = x[0];
#pragma unroll
    for (int i = 1; i < BL_NV; ++i) a += x[i];
    return a;
}

// A row of the workspace: ps [E], c [E] (int), n (int), sum of lse^2; an even number of words.
__host__ __device__ __forceinline__ size_t part_words(int E) { return 2 * (size_t)E + 2; }

// ws: ticket of the second launch, its jobs' values [S * blocks], n [S], sums of lse^2 [S], rows.
struct BlSpace {
    uint32_t* ticket;
    float* value;
    int32_t* n;
    float* z;
    float* part;
};

template <int LPT, bool VEC>
__global__ void __launch_bounds__(BL_THREADS, 1)
    balance_kernel(BlShape s, const float* logits, const int32_t* idx, float* lse_out, float2* kept, BlSpace w) {
    constexpr int TPW = 32 / LPT;  // tokens of a warp
    __shared__ float psum[BL_WARPS][BL_MAX_E];
    __shared__ int cnt[BL_MAX_E];
    __shared__ float zsum[BL_WARPS];
    __shared__ int nsum[BL_WARPS];
    griddep_wait();
    griddep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, lig = lane % LPT, tig = lane / LPT;
    if (blockIdx.x == 0 && tid == 0) *w.ticket = 0;
    int pos = blockIdx.x * s.chunk;
    const int last = min(s.T, pos + s.chunk);
    for (int seq = sequence_of(s, pos); pos < last && seq <= s.S; ++seq) {
        const int end = min(last, seq < 0 ? start_of(s, 0) : seq < s.S ? start_of(s, seq + 1) : s.T);
        if (end <= pos) continue;
        const bool counted = seq >= 0 && seq < s.S;
        for (int e = tid; e < s.E; e += BL_THREADS) cnt[e] = 0;
        __syncthreads();
        float p[BL_NV], z = 0.f;
        int n = 0;
#pragma unroll
        for (int i = 0; i < BL_NV; ++i) p[i] = 0.f;
        // a token's logits, mask and (its first LPT) choices are on their way while the token before is worked on
        float next[BL_NV];
        int next_e = -1;
        bool next_live = false;
        auto fetch = [&](int b) {
            const int t = b + tig;
            const bool there = t < end;
            load_row<LPT, VEC>(logits + (size_t)t * s.E, there, s.E, lig, next);
            next_live = there && counted && (!s.mask || s.mask[t]);
            next_e = there && lig < s.k ? idx[(size_t)t * s.k + lig] : -1;
        };
        fetch(pos + warp * TPW);
#pragma unroll 2
        for (int b = pos + warp * TPW; b < end; b += BL_WARPS * TPW) {
            const int t = b + tig, e0 = next_e;
            const bool there = t < end, live = next_live;
            float x[BL_NV];
#pragma unroll
            for (int i = 0; i < BL_NV; ++i) x[i] = next[i];
            fetch(b + BL_WARPS * TPW);
            const float m = exponentials<LPT>(x), sum = group_sum<LPT>(sum_of(x));
            const float lse = m + __logf(sum);  // (off by 2^-21 at most: sums are at least 1)
            const float inv = sum == 0.f ? 0.f : __fdividef(1.0f, sum);
            if (there && lig == 0) {
                if (lse_out) lse_out[t] = lse;
                if (kept) kept[t] = make_float2(m, inv);
            }
            if (live && sum != 0.f) {
#pragma unroll
                for (int i = 0; i < BL_NV; ++i) p[i] = fmaf(x[i], inv, p[i]);
                if (lig == 0) {
                    z = fmaf(lse, lse, z);
                    ++n;
                }
                if ((unsigned)e0 < (unsigned)s.E) atomicAdd(&cnt[e0], 1);
                for (int j = lig + LPT; j < s.k; j += LPT) {
                    const int e = idx[(size_t)t * s.k + j];
                    if ((unsigned)e < (unsigned)s.E) atomicAdd(&cnt[e], 1);
                }
            }
        }
        if (counted) {
#pragma unroll
            for (int i = 0; i < BL_NV; ++i)
#pragma unroll
                for (int o = LPT; o < 32; o <<= 1) p[i] += __shfl_xor_sync(0xffffffffu, p[i], o);
            z = warp_sum(z);
            n = __reduce_add_sync(0xffffffffu, n);
            if (tig == 0) {
#pragma unroll
                for (int i = 0; i < BL_NV; ++i) {
                    const int c = column<LPT, VEC>(lig, i);
                    if (c < s.E) psum[warp][c] = p[i];
                }
            }
            if (lane == 0) {
                zsum[warp] = z;
                nsum[warp] = n;
            }
            __syncthreads();
            float* row = w.part + (size_t)(blockIdx.x + seq) * part_words(s.E);
            for (int e = tid; e < s.E; e += BL_THREADS) {
                float a = 0.f;
#pragma unroll
                for (int i = 0; i < BL_WARPS; ++i) a += psum[i][e];
                row[e] = a;
                reinterpret_cast<int32_t*>(row)[s.E + e] = cnt[e];
            }
            if (warp == 0) {
                z = warp_sum(zsum[lane]);
                n = __reduce_add_sync(0xffffffffu, nsum[lane]);
                if (lane == 0) {
                    reinterpret_cast<int32_t*>(row)[2 * s.E] = n;
                    row[2 * s.E + 1] = z;
                }
            }
            __syncthreads();
        }
        pos = end;
    }
}

// What balance_backward reads: w_b / S', 2 w_z / N, a [S, E] without the 1 / S'.
constexpr int BL_SAVED_HEAD = 4;  // floats
// Behind them, each token's largest logit and 1 / sum of exp(l - that) (0 for a token without probabilities).
__host__ __device__ __forceinline__ size_t kept_at(int S, int E) { return (BL_SAVED_HEAD + (size_t)S * E + 1) / 2 * 2; }  // floats

struct BlEnd {
    int blocks, splits;  // blocks of 32 columns of a row; warps that share a job (a sequence's block), a power of two
    float wb, wz;
    float* loss;
    int32_t* counts;
    float* saved;
};

__global__ void __launch_bounds__(BL_END_WARPS * 32) balance_end_kernel(BlShape s, BlSpace w, BlEnd f) {
    __shared__ float ps[BL_END_WARPS][32], zs[BL_END_WARPS];
    __shared__ int cs[BL_END_WARPS][32], ns[BL_END_WARPS];
    __shared__ bool am_last;
    griddep_wait();
    griddep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, split = warp & (f.splits - 1), warps = blockDim.x >> 5;
    const int jobs = s.S * f.blocks, per = warps / f.splits;
    const size_t words = part_words(s.E);
    for (int j0 = blockIdx.x * per; j0 < jobs; j0 += gridDim.x * per) {
        const int job = j0 + warp / f.splits;
        const int seq = job / f.blocks, c = (job - seq * f.blocks) * 32 + lane;
        float a = 0.f, z = 0.f;
        int k = 0, n = 0;
        if (job < jobs) {
            const int from = start_of(s, seq), to = start_of(s, seq + 1);
            if (to > from) {
                const int end = (to - 1) / s.chunk;
                for (int b = from / s.chunk + split; b <= end; b += 8 * f.splits) {  // eight rows in flight
                    float va[8], vz[8];
                    int vk[8], vn[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const bool there = b + i * f.splits <= end;
                        const float* row = w.part + (size_t)(b + i * f.splits + seq) * words;
                        const int32_t* irow = reinterpret_cast<const int32_t*>(row);
                        va[i] = there && c < s.E ? row[c] : 0.f;
                        vk[i] = there && c < s.E ? irow[s.E + c] : 0;
                        vn[i] = there ? irow[2 * s.E] : 0;
                        vz[i] = there ? row[2 * s.E + 1] : 0.f;
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        a += va[i];
                        k += vk[i];
                        n += vn[i];
                        z += vz[i];
                    }
                }
            }
        }
        ps[warp][lane] = a;
        cs[warp][lane] = k;
        if (lane == 0) {
            ns[warp] = n;
            zs[warp] = z;
        }
        __syncthreads();
        if (split == 0 && job < jobs) {
            for (int i = 1; i < f.splits; ++i) {
                a += ps[warp + i][lane];
                k += cs[warp + i][lane];
                n += ns[warp + i];
                z += zs[warp + i];
            }
            const float slope = n ? (float)k * ((float)s.E / ((float)s.k * (float)n * (float)n)) : 0.f;
            if (c < s.E) {
                f.counts[(size_t)seq * s.E + c] = k;
                if (f.saved) f.saved[BL_SAVED_HEAD + (size_t)seq * s.E + c] = slope;
            }
            const float v = warp_sum(slope * a);
            if (lane == 0) {
                w.value[job] = v;
                if (c < 32) {
                    w.n[seq] = n;
                    w.z[seq] = z;
                }
            }
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        __threadfence();
        am_last = atomicAdd(w.ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!am_last) return;
    __threadfence();
    float v = 0.f, z = 0.f;
    int n = 0, used = 0;
    for (int i = threadIdx.x; i < jobs; i += blockDim.x) v += __ldcg(w.value + i);
    for (int i = threadIdx.x; i < s.S; i += blockDim.x) {
        const int k = __ldcg(w.n + i);
        z += __ldcg(w.z + i);
        n += k;
        used += k > 0;
    }
    v = warp_sum(v);
    z = warp_sum(z);
    n = __reduce_add_sync(0xffffffffu, n);
    used = __reduce_add_sync(0xffffffffu, used);
    if (lane == 0) {
        ps[warp][0] = v;
        zs[warp] = z;
        ns[warp] = n;
        cs[warp][0] = used;
    }
    __syncthreads();
    if (warp) return;
    const bool mine = lane < warps;
    v = warp_sum(mine ? ps[lane][0] : 0.f);
    z = warp_sum(mine ? zs[lane] : 0.f);
    n = __reduce_add_sync(0xffffffffu, mine ? ns[lane] : 0);
    used = __reduce_add_sync(0xffffffffu, mine ? cs[lane][0] : 0);
    if (lane) return;
    const float bal = used ? v / (float)used : 0.f, zl = n ? z / (float)n : 0.f;
    // (a loss without weight leaves the sum alone, infinite or not)
    f.loss[0] = (f.wb != 0.f ? f.wb * bal : 0.f) + (f.wz != 0.f ? f.wz * zl : 0.f);
    f.loss[1] = bal;
    f.loss[2] = zl;
    if (f.saved) {
        f.saved[0] = used ? f.wb / (float)used : 0.f;
        f.saved[1] = n ? 2.f * f.wz / (float)n : 0.f;
    }
}

template <int LPT, bool VEC>
__global__ void __launch_bounds__(BL_BACK_THREADS, BL_BACK_CTAS)
    balance_backward_kernel(BlShape s, const float* logits, const int32_t* idx, const float* saved, const float* gates,
                            const float* dgates, const float* dloss, float* dlogits) {
    constexpr int TPW = 32 / LPT;
    __shared__ __align__(16) float rows[BL_BACK_WARPS][32 * BL_NV];
    griddep_wait();
    griddep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, lig = lane % LPT, tig = lane / LPT;
    const int first = blockIdx.x * s.chunk, last = min(s.T, first + s.chunk);
    const float up = dloss ? *dloss : 1.0f, wb = saved[0] * up, wz = saved[1] * up;
    const float* slopes = saved + BL_SAVED_HEAD;
    const float2* kept = reinterpret_cast<const float2*>(saved + kept_at(s.S, s.E));
    int seq = -2, seq_end = 0;  // this lane's token's, and where it ends
    float a[BL_NV], next[BL_NV];
#pragma unroll
    for (int i = 0; i < BL_NV; ++i) a[i] = 0.f;
    // a token's logits, mask and (its first LPT) pairs are on their way while the token before is worked on
    int next_e = -1;
    float next_g = 0.f, next_d = 0.f;
    float2 next_kept = make_float2(0.f, 0.f);
    bool next_live = false;
    auto fetch = [&](int b) {
        const int t = b + tig;
        const bool there = t < last;
        load_row<LPT, VEC>(logits + (size_t)t * s.E, there, s.E, lig, next);
        next_live = there && (!s.mask || s.mask[t]);
        if (there) next_kept = kept[t];
        if (gates) {
            const bool pair = there && lig < s.k;
            const size_t at = (size_t)t * s.k + lig;
            next_e = pair ? idx[at] : -1;
            next_g = pair ? gates[at] : 0.f;
            next_d = pair ? dgates[at] : 0.f;
        }
    };
    float* const mine = rows[warp] + tig * (BL_NV * LPT);  // the token's row, for the gates' part
    fetch(first + warp * TPW);
#pragma unroll 1
    for (int b = first + warp * TPW; b < last; b += BL_BACK_WARPS * TPW) {
        const int t = b + tig, e0 = next_e;
        const bool there = t < last;
        const float g0 = next_g, d0 = next_d;
        const float m = next_kept.x, inv = next_kept.y;
        bool live = next_live;
        float x[BL_NV];
#pragma unroll
        for (int i = 0; i < BL_NV; ++i) x[i] = next[i];
        fetch(b + BL_BACK_WARPS * TPW);
        if (there && (seq == -2 || t >= seq_end)) {
            seq = sequence_of(s, t);
            seq_end = seq < 0 ? start_of(s, 0) : seq < s.S ? start_of(s, seq + 1) : s.T;
#pragma unroll
            for (int i = 0; i < BL_NV; ++i) {
                const int c = column<LPT, VEC>(lig, i);
                a[i] = seq >= 0 && seq < s.S && c < s.E ? slopes[(size_t)seq * s.E + c] : 0.f;
            }
        }
        float dot = 0.f, gd = g0 * d0;
#pragma unroll
        for (int i = 0; i < BL_NV; ++i) {
            x[i] = exponential(x[i] - m);
            dot = fmaf(x[i], a[i], dot);
        }
        if (gates) {
            for (int j = lig + LPT; j < s.k; j += LPT)
                if (there) gd = fmaf(gates[(size_t)t * s.k + j], dgates[(size_t)t * s.k + j], gd);
        }
        group_sums<LPT>(dot, gd, lane);
        live = live && seq >= 0 && seq < s.S && inv != 0.f;
        const float zl = wz * (m - __logf(inv));
        dot *= inv;
#pragma unroll
        for (int i = 0; i < BL_NV; ++i) x[i] = live ? x[i] * inv * fmaf(wb, a[i] - dot, zl) : 0.f;
        if (gates) {
            // through shared memory, where a pair's value finds its expert's place; pairs of one token that name the
            // same expert go one after another
#pragma unroll
            for (int i = 0; i < BL_NV; i += 4) {
                if (VEC) {
                    *reinterpret_cast<float4*>(mine + column<LPT, VEC>(lig, i)) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) mine[column<LPT, VEC>(lig, i + k)] = x[i + k];
                }
            }
            __syncwarp();
            for (int j0 = 0; j0 < s.k; j0 += LPT) {
                const int j = j0 + lig;
                const size_t at = (size_t)t * s.k + j;
                const bool pair = live && j < s.k;
                const int e = j0 == 0 ? e0 : pair ? idx[at] : -1;
                const float v = j0 == 0 ? g0 * (d0 - gd) : pair ? gates[at] * (dgates[at] - gd) : 0.f;
                const bool good = pair && (unsigned)e < (unsigned)s.E;
                if (LPT == 1) {
                    if (good) mine[e] += v;
                } else {
                    const uint32_t same = __match_any_sync(0xffffffffu, good ? tig * BL_MAX_E + e : -1 - lane);
                    if (__any_sync(0xffffffffu, same & (same - 1))) {
                        for (int k = 0; k < LPT; ++k) {
                            if (good && lig == k) mine[e] += v;
                            __syncwarp();
                        }
                    } else if (good) {
                        mine[e] += v;
                    }
                }
                __syncwarp();
            }
#pragma unroll
            for (int i = 0; i < BL_NV; i += 4) {
                if (VEC) {
                    const float4 v = *reinterpret_cast<const float4*>(mine + column<LPT, VEC>(lig, i));
                    x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[i + k] = mine[column<LPT, VEC>(lig, i + k)];
                }
            }
            __syncwarp();
        }
        if (!there) continue;
        float* row = dlogits + (size_t)t * s.E;
        if (VEC) {
#pragma unroll
            for (int q = 0; q < BL_NV / 4; ++q) {
                const int c = (q * LPT + lig) * 4;
                if (c < s.E) *reinterpret_cast<float4*>(row + c) = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < BL_NV; ++i) {
                const int c = i * LPT + lig;
                if (c < s.E) row[c] = x[i];
            }
        }
    }
}

int check(const moe_balance_config* c) {
    if (!c) return fail(MOE_ERR_ARG, "config is NULL");
    if (c->T < 0 || c->T >= 1 << 24) return fail(MOE_ERR_ARG, "T=%d must be in [0, 2^24)", c->T);
    if (c->E < 1 || c->E > BL_MAX_E) return fail(MOE_ERR_ARG, "E=%d must be in [1, %d]", c->E, BL_MAX_E);
    if (c->topk < 1 || c->topk > BL_MAX_K) return fail(MOE_ERR_ARG, "topk=%d must be in [1, %d]", c->topk, BL_MAX_K);
    if (c->seqs < 1 || c->seqs >= 1 << 24) return fail(MOE_ERR_ARG, "seqs=%d must be in [1, 2^24)", c->seqs);
    if (!isfinite(c->balance) || !isfinite(c->z))
        return fail(MOE_ERR_ARG, "balance=%g and z=%g must be finite", (double)c->balance, (double)c->z);
    for (int i = 0; i < 4; ++i)
        if (c->reserved[i]) return fail(MOE_ERR_ARG, "reserved fields must be zero");
    return MOE_OK;
}

int lanes_of(int E) {  // of a token
    int l = 1;
    while (l * BL_NV < E) l *= 2;
    return l;
}
int ctas_of(const moe_balance_config& c, int threads, int most) {
    const int pass = threads / lanes_of(c.E);  // tokens that a CTA has in its registers at once
    const int n = (c.T + pass - 1) / pass;
    return n < 1 ? 1 : n < most ? n : most;
}
int most_ctas(const DeviceInfo& di) { return di.sms < BL_MAX_CTAS ? di.sms : BL_MAX_CTAS; }

BlShape shape_of(const moe_balance_config& c, const int32_t* offsets, const uint8_t* mask, int ctas) {
    BlShape s;
    s.T = c.T, s.E = c.E, s.k = c.topk, s.S = c.seqs;
    s.chunk = c.T ? (c.T + ctas - 1) / ctas : 1;
    s.ctas = ctas;
    s.offsets = offsets;
    s.mask = mask;
    return s;
}

size_t blocks_of(int E) { return ((size_t)E + 31) / 32; }
size_t space_bytes(const moe_balance_config& c, int ctas) {
    return 256 + align_up(4 * (size_t)c.seqs * (blocks_of(c.E) + 2), 16) + 4 * part_words(c.E) * ((size_t)ctas + c.seqs);
}
BlSpace space_of(const moe_balance_config& c, void* ws) {
    BlSpace w;
    char* p = static_cast<char*>(ws);
    w.ticket = reinterpret_cast<uint32_t*>(p);
    w.value = reinterpret_cast<float*>(p + 256);
    w.n = reinterpret_cast<int32_t*>(w.value + (size_t)c.seqs * blocks_of(c.E));
    w.z = reinterpret_cast<float*>(w.n + c.seqs);
    w.part = reinterpret_cast<float*>(p + 256 + align_up(4 * (size_t)c.seqs * (blocks_of(c.E) + 2), 16));
    return w;
}

// f(lanes of a token, whole vectors?) for the config.
template <typename F>
cudaError_t dispatch(int E, bool vec, F f) {
    auto on = [&](auto lpt) { return vec ? f(lpt, std::true_type()) : f(lpt, std::false_type()); };
    switch (lanes_of(E)) {
        case 1: return on(Int<1>());
        case 2: return on(Int<2>());
        case 4: return on(Int<4>());
        case 8: return on(Int<8>());
        case 16: return on(Int<16>());
        default: return on(Int<32>());
    }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

MOE_API int moe_balance_workspace_size(const moe_balance_config* c, size_t* bytes) {
    clear_error();
    const int rc = check(c);
    if (rc) return rc;
    if (!bytes) return fail(MOE_ERR_ARG, "bytes is NULL");
    *bytes = space_bytes(*c, ctas_of(*c, BL_THREADS, BL_MAX_CTAS));
    return MOE_OK;
}

MOE_API int moe_balance_saved_size(const moe_balance_config* c, size_t* bytes) {
    clear_error();
    const int rc = check(c);
    if (rc) return rc;
    if (!bytes) return fail(MOE_ERR_ARG, "bytes is NULL");
    *bytes = 4 * (kept_at(c->seqs, c->E) + 2 * (size_t)c->T);
    return MOE_OK;
}

MOE_API int moe_balance_forward(const moe_balance_config* c, const float* logits, const int32_t* idx,
                                const int32_t* offsets, const uint8_t* mask, float* loss, int32_t* counts, float* lse,
                                void* saved, void* ws, size_t ws_bytes, void* stream) {
    clear_error();
    int rc = check(c);
    if (rc) return rc;
    if (!offsets && c->seqs != 1) return fail(MOE_ERR_ARG, "seqs=%d needs offsets", c->seqs);
    if ((c->T && (!logits || !idx)) || !loss || !counts || !ws) return fail(MOE_ERR_ARG, "NULL input, output or workspace");
    if (!aligned(logits, 4) || !aligned(idx, 4) || !aligned(offsets, 4) || !aligned(loss, 4) || !aligned(counts, 4) ||
        !aligned(lse, 4) || !aligned(saved, 16) || !aligned(ws, 16))
        return fail(MOE_ERR_ARG, "a pointer is not aligned (saved and ws to 16 bytes, the others to their type)");
    DeviceInfo di;
    if ((rc = check_device(&di))) return rc;
    const int ctas = ctas_of(*c, BL_THREADS, most_ctas(di));
    const size_t need = space_bytes(*c, ctas);
    if (ws_bytes < need) return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
    const BlShape s = shape_of(*c, offsets, mask, ctas);
    const BlSpace w = space_of(*c, ws);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = dispatch(c->E, c->E % 4 == 0 && aligned(logits, 16), [&](auto lpt, auto vec) {
        return launch_k(balance_kernel<decltype(lpt)::value, decltype(vec)::value>, dim3(ctas), dim3(BL_THREADS), 0, st, true,
                        s, logits, idx, lse, saved ? reinterpret_cast<float2*>(static_cast<float*>(saved) + kept_at(c->seqs, c->E)) : nullptr, w);
    });
    if (e != cudaSuccess) return cuda_fail(e, "balance loss launch");
    BlEnd f;
    f.blocks = (int)blocks_of(c->E);
    f.wb = c->balance, f.wz = c->z;
    f.loss = loss, f.counts = counts, f.saved = static_cast<float*>(saved);
    // as many warps on a job as it has rows on average, up to a CTA's
    f.splits = 1;
    while (f.splits < BL_END_WARPS && f.splits < (ctas + c->seqs - 1) / c->seqs) f.splits *= 2;
    const int warps = f.splits < 8 ? 8 : f.splits, jobs = c->seqs * f.blocks, per = warps / f.splits, n = (jobs + per - 1) / per;
    e = launch_k(balance_end_kernel, dim3(n < 4 * di.sms ? n : 4 * di.sms), dim3(warps * 32), 0, st, true, s, w, f);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "balance loss launch");
}

MOE_API int moe_balance_backward(const moe_balance_config* c, const float* logits, const int32_t* idx,
                                 const int32_t* offsets, const uint8_t* mask, const void* saved, const float* gates,
                                 const float* dgates, const float* dloss, float* dlogits, void* stream) {
    clear_error();
    int rc = check(c);
    if (rc) return rc;
    if (!offsets && c->seqs != 1) return fail(MOE_ERR_ARG, "seqs=%d needs offsets", c->seqs);
    if (!gates != !dgates) return fail(MOE_ERR_ARG, "gates and dgates go together");
    if (c->T == 0) return MOE_OK;
    if (!logits || !idx || !saved || !dlogits) return fail(MOE_ERR_ARG, "NULL input or output pointer");
    if (!aligned(logits, 4) || !aligned(idx, 4) || !aligned(offsets, 4) || !aligned(gates, 4) || !aligned(dgates, 4) ||
        !aligned(dloss, 4) || !aligned(dlogits, 4) || !aligned(saved, 16))
        return fail(MOE_ERR_ARG, "a pointer is not aligned (saved to 16 bytes, the others to their type)");
    DeviceInfo di;
    if ((rc = check_device(&di))) return rc;
    const int ctas = ctas_of(*c, BL_BACK_THREADS, BL_BACK_CTAS * di.sms);
    const BlShape s = shape_of(*c, offsets, mask, ctas);
    const bool vec = c->E % 4 == 0 && aligned(logits, 16) && aligned(dlogits, 16);
    const cudaError_t e = dispatch(c->E, vec, [&](auto lpt, auto v) {
        return launch_k(balance_backward_kernel<decltype(lpt)::value, decltype(v)::value>, dim3(ctas), dim3(BL_BACK_THREADS), 0,
                        static_cast<cudaStream_t>(stream), true, s, logits, idx, static_cast<const float*>(saved), gates,
                        dgates, dloss, dlogits);
    });
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "balance loss backward launch");
}

}  // extern "C"
