// Balance loss and z loss of a router with the experts' loads, and the gradient of its logits.
//
//   p = softmax(l), lse = log sum exp(l); of sequence s: n tokens, c[e] pairs, ps[e] = sum of p
//   balance = mean over sequences with n > 0 of E / (k n^2) sum_e c[e] ps[e],  z = mean over tokens of lse^2
//   dl = dloss p (w_b / S' (a - sum_e p a) + 2 w_z / N lse) + the gates' part,  a[e] = E / (k n^2) c[e]
//
// The logits are read once in each direction and dlogits written once: HBM traffic bounds both passes. A row lies in
// the registers of as many lanes as hold it with eight values a lane (of 16 lanes with sixteen beyond 128 experts), so a
// warp works on 2 to 32 tokens at once.
// Forward: a CTA takes consecutive tokens and keeps its sums of p in registers until the sequence ends; counts
// are integers in shared memory. What it has of a sequence goes to a row of the workspace: CTA and sequence both
// grow along the tokens, so the pair's rank is their sum. A second launch adds the rows up in the order of the
// CTAs (no sum depends on which CTA was first) and its last CTA makes the losses.
// Times here are those of calls that run one behind the other on the device. 131072 tokens of 256 experts in 67 sequences: 90 us
// for both passes (402 MB with the second read of the logits, 4.5 TB/s; issue slots 54 to 63 % used). 16384 tokens of 64
// experts: 15 us; 4096 of 8, forward: 6.7 us, two dependent launches.
#include <math.h>

#include "row_values.cuh"

namespace moe {
namespace {

constexpr int BL_THREADS = 768, BL_WARPS = BL_THREADS / 32;       // forward: one CTA a SM, so few rows of sums
constexpr int BL_BACK_THREADS = 256, BL_BACK_WARPS = BL_BACK_THREADS / 32, BL_BACK_CTAS = 3;
constexpr int BL_MAX_CTAS = 1024;  // of the forward pass
constexpr int BL_MAX_E = 256, BL_MAX_K = 8;
constexpr int BL_END_WARPS = 32;   // of the second launch's CTAs, at most

struct BlShape {
    int T, E, k, S, chunk;  // a CTA takes `chunk` consecutive tokens
    const int32_t* offsets;
    const uint8_t* mask;
};
// Where sequence i starts (i = S: where the last one ends), within [0, T] whatever the caller's array holds. Up to
// BL_STARTS - 1 sequences' starts are fetched at once into shared memory: a search through global memory is a chain
// of waits.
constexpr int BL_STARTS = 256;
struct BlStarts {
    const int32_t* in;  // clamped, in shared memory, or null
    __device__ __forceinline__ BlStarts(const BlShape& s, int32_t* space) : in(nullptr) {
        if (!s.offsets || s.S >= BL_STARTS) return;
        for (int i = threadIdx.x; i <= s.S; i += blockDim.x) space[i] = min(max(s.offsets[i], 0), s.T);
        __syncthreads();
        in = space;
    }
    __device__ __forceinline__ int operator()(const BlShape& s, int i) const {
        if (in) return in[i];
        if (!s.offsets) return i == 0 ? 0 : s.T;
        return min(max(s.offsets[i], 0), s.T);
    }
    // The sequence of token t: -1 before the first, S behind the last.
    __device__ __forceinline__ int find(const BlShape& s, int t) const {
        if (!s.offsets) return t < s.T ? 0 : 1;
        if (t < (*this)(s, 0)) return -1;
        int lo = 0, hi = s.S;  // the last one that starts at or before t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((*this)(s, mid) <= t) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    }
};

// Column of a lane's value i: four neighbours (float4 loads) or every LPT-th.
template <int LPT, bool VEC>
__device__ __forceinline__ int column(int lig, int i) {
    return VEC ? ((i >> 2) * LPT + lig) * 4 + (i & 3) : i * LPT + lig;
}
// A warp's tokens' logits lie side by side in memory, 32 NV of them at most. They come through a ring of BL_DEPTH places
// of the warp's own in shared memory, fetched by cp.async that many steps ahead: one step held in registers left the
// memory waiting (few bytes in flight).
constexpr int BL_DEPTH = 3;
template <int PLACE, bool VEC>
__device__ __forceinline__ void fetch_rows(float* to, const float* from, int n, int lane) {
    if (VEC) {
#pragma unroll
        for (int k = 0; k < PLACE / 128; ++k)
            if ((lane + 32 * k) * 4 < n) copy_async<16>(to + (lane + 32 * k) * 4, from + (lane + 32 * k) * 4);
    } else {
#pragma unroll
        for (int k = 0; k < PLACE / 32; ++k)
            if (lane + 32 * k < n) copy_async<4>(to + lane + 32 * k, from + lane + 32 * k);
    }
}
template <int N>
__device__ __forceinline__ void fetched() {  // all but the last N groups
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// A lane's values of a row, two and two; -inf where there is none.
template <int LPT, bool VEC, int N2>
__device__ __forceinline__ void load_row(const float* row, bool there, int E, int lig, f2 (&x)[N2]) {
    if (VEC) {
#pragma unroll
        for (int q = 0; q < N2 / 2; ++q) {
            const int c = (q * LPT + lig) * 4;
            float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (there && c < E) v = *reinterpret_cast<const float4*>(row + c);
            x[2 * q] = pair(v.x, v.y);
            x[2 * q + 1] = pair(v.z, v.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N2; ++i) {
            const int c = 2 * i * LPT + lig;
            x[i] = pair(there && c < E ? row[c] : -INFINITY, there && c + LPT < E ? row[c + LPT] : -INFINITY);
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
constexpr float BL_LOG2E = 1.4426950408889634f;
__device__ __forceinline__ float exp2_of(float v) {  // (below 2^-126: zero)
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// x becomes exp(x - m). By one product and sum: what m's product with log2(e) is rounded by (2^-14 at most up to BL_FAR) is
// a factor of the whole row, which its sum takes out again, and which leaves a row's largest value within 2^-14 of 1. In
// rows beyond (from 2^31 on that factor itself could leave fp32's range) the difference is taken first.
constexpr float BL_FAR = 1024.f;
template <int N2>
__device__ __forceinline__ void exponentials(f2 (&x)[N2], float m) {
    const bool far = fabsf(m) > BL_FAR;
    const f2 l = both<f2>(BL_LOG2E), c = both<f2>(far ? 0.f : -m * BL_LOG2E);
    if (far) {
#pragma unroll
        for (int i = 0; i < N2; ++i) x[i] = add_(x[i], both<f2>(-m));
    }
#pragma unroll
    for (int i = 0; i < N2; ++i) {
        const float2 v = split(fma_(x[i], l, c));
        x[i] = pair(exp2_of(v.x), exp2_of(v.y));
    }
}
// The row's largest value, 0 if every one is -inf.
template <int LPT, int N2>
__device__ __forceinline__ float largest(const f2 (&x)[N2]) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < N2; ++i) {
        const float2 v = split(x[i]);
        m = fmaxf(m, fmaxf(v.x, v.y));
    }
#pragma unroll
    for (int o = LPT / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m == -INFINITY ? 0.f : m;
}
template <int N2>
__device__ __forceinline__ float sum_of(const f2 (&x)[N2]) {
    f2 a = x[0];
#pragma unroll
    for (int i = 1; i < N2; ++i) a = add_(a, x[i]);
    return total(a);
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

// What balance_backward reads: w_b / S', 2 w_z / N, a [S, E] without the 1 / S'.
constexpr int BL_SAVED_HEAD = 4;  // floats
// Behind them, of each token the largest logit, 1 / sum of exp(l - that) (0 for a token without probabilities) and lse (from
// the inverse it would carry that one's rounding as well, which is much of an lse next to zero, and cost a logarithm).
struct BlKept {
    float m, inv, lse;
};
__host__ __device__ __forceinline__ size_t kept_at(int S, int E) { return BL_SAVED_HEAD + (size_t)S * E; }  // floats

template <int LPT, int NV, bool VEC>
__global__ void __launch_bounds__(BL_THREADS, 1)
    balance_kernel(BlShape s, const float* logits, const int32_t* idx, float* lse_out, BlKept* kept, BlSpace w) {
    constexpr int TPW = 32 / LPT, N2 = NV / 2, PLACE = 32 * NV;  // tokens of a warp, a lane's pairs of logits, floats of a place
    extern __shared__ __align__(16) float bl_smem[];  // [warps][BL_DEPTH][PLACE]; at a sequence's end sums [warps][256]
    __shared__ int cnt[BL_MAX_E];
    __shared__ float zsum[BL_WARPS];
    __shared__ int nsum[BL_WARPS];
    griddep_wait();
    griddep_launch();
    __shared__ int32_t starts_space[BL_STARTS];
    const BlStarts starts(s, starts_space);
    const int tid = threadIdx.x, warps = blockDim.x >> 5, warp = tid >> 5, lane = tid & 31, lig = lane % LPT, tig = lane / LPT;
    float* const ring = bl_smem + warp * (BL_DEPTH * PLACE);
    if (blockIdx.x == 0 && tid == 0) *w.ticket = 0;
    int pos = blockIdx.x * s.chunk;
    const int last = min(s.T, pos + s.chunk);
    for (int seq = starts.find(s, pos); pos < last && seq <= s.S; ++seq) {
        const int end = min(last, seq < 0 ? starts(s, 0) : seq < s.S ? starts(s, seq + 1) : s.T);
        if (end <= pos) {  // past all empty sequences at once
            seq = max(seq, starts.find(s, pos) - 1);
            continue;
        }
        const bool counted = seq >= 0 && seq < s.S;
        for (int e = tid; e < s.E; e += blockDim.x) cnt[e] = 0;
        __syncthreads();
        f2 p[N2];
        float z = 0.f;
        int n = 0;
#pragma unroll
        for (int i = 0; i < N2; ++i) p[i] = both<f2>(0.f);
        // a token's mask and (its first LPT) choices are two steps ahead of it, its logits BL_DEPTH - 1
        const int step = warps * TPW;
        int e1 = -1, e2 = -1;
        bool live1 = false, live2 = false;
        auto fetch = [&](int t) {
            const bool there = t < end && counted;
            e1 = e2;
            live1 = live2;
            live2 = there && (!s.mask || s.mask[t]);
            e2 = there && lig < s.k ? idx[(size_t)t * s.k + lig] : -1;
        };
        auto issue = [&](int b, float* to) {
            if (b < end) fetch_rows<PLACE, VEC>(to, logits + (size_t)b * s.E, min(TPW, end - b) * s.E, lane);
            committed();
        };
        int t = pos + warp * TPW + tig;
        float* here = ring;
#pragma unroll
        for (int k = 0; k < BL_DEPTH - 1; ++k) issue(t - tig + k * step, ring + k * PLACE);
        fetch(t);
        fetch(t + step);
#pragma unroll 1
        for (; t - tig < end; t += step) {
            const int e0 = e1;
            const bool there = t < end, live = live1;
            fetch(t + 2 * step);
            issue(t - tig + (BL_DEPTH - 1) * step, here == ring ? ring + (BL_DEPTH - 1) * PLACE : here - PLACE);
            fetched<BL_DEPTH - 1>();
            __syncwarp();
            f2 x[N2];
            load_row<LPT, VEC>(here + tig * s.E, there, s.E, lig, x);
            here = here == ring + (BL_DEPTH - 1) * PLACE ? ring : here + PLACE;
            __syncwarp();
            const float m = largest<LPT>(x);
            exponentials(x, m);
            const float sum = group_sum<LPT>(sum_of(x));
            // logf: an lse next to zero is the logarithm of a sum next to 1, where __logf is off by 2^-21 (131072 tokens of 256
            // experts, both passes: 90.1 us; 89.3 with __logf). The inverse is off by 2 units in the last place, as every
            // exponential that it multiplies is (2000 tokens of 64 experts in 100 sequences: 17.5 us; 18.2 with a division).
            const float lse = m + logf(sum);
            const float inv = sum == 0.f ? 0.f : __fdividef(1.0f, sum);
            if (there && lig == 0) {
                if (lse_out) lse_out[t] = lse;
                if (kept) kept[t] = BlKept{m, inv, lse};
            }
            if (live && sum != 0.f) {
                const f2 v = both<f2>(inv);
#pragma unroll
                for (int i = 0; i < N2; ++i) p[i] = fma_(x[i], v, p[i]);
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
        fetched<0>();
        __syncwarp();
        if (counted) {
            float v[NV];
#pragma unroll
            for (int i = 0; i < N2; ++i) {
                const float2 e = split(p[i]);
                v[2 * i] = e.x;
                v[2 * i + 1] = e.y;
            }
            // over the warp's tokens: at each step a lane hands half of its columns over and keeps the other half
            int kept_from = 0;
            bool writer = true;
#pragma unroll
            for (int o = LPT, n = NV; o < 32; o <<= 1) {
                const bool hi = lane & o;
                if (n > 1) {
                    n /= 2;
#pragma unroll
                    for (int i = 0; i < n; ++i) {
                        const float send = hi ? v[i] : v[i + n], keep = hi ? v[i + n] : v[i];
                        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                    }
                    kept_from += hi ? n : 0;
                } else {
                    v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
                    writer = writer && !hi;
                }
            }
            z = warp_sum(z);
            n = __reduce_add_sync(0xffffffffu, n);
            constexpr int LEFT = NV > TPW ? NV / TPW : 1;
            if (writer) {
#pragma unroll
                for (int i = 0; i < LEFT; ++i) {
                    const int c = column<LPT, VEC>(lig, kept_from + i);
                    if (c < s.E) ring[c] = v[i];
                }
            }
            if (lane == 0) {
                zsum[warp] = z;
                nsum[warp] = n;
            }
            __syncthreads();
            float* row = w.part + (size_t)(blockIdx.x + seq) * part_words(s.E);
            for (int e = tid; e < s.E; e += blockDim.x) {
                float a = 0.f;
#pragma unroll 8
                for (int i = 0; i < warps; ++i) a += bl_smem[i * (BL_DEPTH * PLACE) + e];
                row[e] = a;
                reinterpret_cast<int32_t*>(row)[s.E + e] = cnt[e];
            }
            if (warp == 0) {
                z = warp_sum(lane < warps ? zsum[lane] : 0.f);
                n = __reduce_add_sync(0xffffffffu, lane < warps ? nsum[lane] : 0);
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
    __shared__ int32_t starts_space[BL_STARTS];
    const BlStarts starts(s, starts_space);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, split = warp & (f.splits - 1), warps = blockDim.x >> 5;
    const int jobs = s.S * f.blocks, per = warps / f.splits;
    const size_t words = part_words(s.E);
    for (int j0 = blockIdx.x * per; j0 < jobs; j0 += gridDim.x * per) {
        const int job = j0 + warp / f.splits;
        const int seq = job / f.blocks, c = (job - seq * f.blocks) * 32 + lane;
        float a = 0.f, z = 0.f;
        int k = 0, n = 0;
        if (job < jobs) {
            const int from = starts(s, seq), to = starts(s, seq + 1);
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
#pragma unroll 8
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
    if (gridDim.x > 1) {
        if (threadIdx.x == 0) {
            __threadfence();
            am_last = atomicAdd(w.ticket, 1u) == gridDim.x - 1;
        }
        __syncthreads();
        if (!am_last) return;
        __threadfence();
    }
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

template <int LPT, int NV, bool VEC>
__global__ void __launch_bounds__(BL_BACK_THREADS, BL_BACK_CTAS)
    balance_backward_kernel(BlShape s, const float* logits, const int32_t* idx, const float* saved, const float* gates,
                            const float* dgates, const float* dloss, float* dlogits) {
    constexpr int TPW = 32 / LPT, N2 = NV / 2, PLACE = 32 * NV;
    extern __shared__ __align__(16) float bl_smem[];  // [warps][BL_DEPTH][PLACE]
    griddep_wait();
    griddep_launch();
    __shared__ int32_t starts_space[BL_STARTS];
    const BlStarts starts(s, starts_space);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, lig = lane % LPT, tig = lane / LPT;
    const int first = blockIdx.x * s.chunk, last = min(s.T, first + s.chunk);
    const float up = dloss ? *dloss : 1.0f, wb = saved[0] * up, wz = saved[1] * up;  // dloss's factor in both
    const float* slopes = saved + BL_SAVED_HEAD;
    const BlKept* kept = reinterpret_cast<const BlKept*>(saved + kept_at(s.S, s.E));
    int seq = -2, seq_end = 0;  // this lane's token's, and where it ends
    bool seq_live = false;
    f2 a[N2];  // w_b / S' times the slopes
#pragma unroll
    for (int i = 0; i < N2; ++i) a[i] = both<f2>(0.f);
    // what a token needs beside its logits, with its first LPT pairs, is two steps ahead of it, the logits BL_DEPTH - 1
    const int step = BL_BACK_WARPS * TPW;
    float* const ring = bl_smem + warp * (BL_DEPTH * PLACE);
    struct Small {
        int e = -1;
        float g = 0.f, d = 0.f;
        BlKept kept = {0.f, 0.f, 0.f};
        bool live = false;
    } one, two;
    auto fetch = [&](int t) {
        const bool there = t < last;
        one = two;
        two.live = there && (!s.mask || s.mask[t]);
        if (there) two.kept = kept[t];
        if (gates && there && lig < s.k) {
            const size_t at = (size_t)t * s.k + lig;
            two.e = idx[at];
            two.g = gates[at];
            two.d = dgates[at];
        }
    };
    auto issue = [&](int b, float* to) {
        if (b < last) fetch_rows<PLACE, VEC>(to, logits + (size_t)b * s.E, min(TPW, last - b) * s.E, lane);
        committed();
    };
    int t = first + warp * TPW + tig;
    float* here = ring;
#pragma unroll
    for (int k = 0; k < BL_DEPTH - 1; ++k) issue(t - tig + k * step, ring + k * PLACE);
    fetch(t);
    fetch(t + step);
#pragma unroll 1
    for (; t - tig < last; t += step) {
        const int e0 = one.e;
        const bool there = t < last;
        const float g0 = one.g, d0 = one.d, m = one.kept.m, inv = one.kept.inv, lse = one.kept.lse;
        bool live = one.live;
        const size_t at = (size_t)t * s.k + lig;
        fetch(t + 2 * step);
        issue(t - tig + (BL_DEPTH - 1) * step, here == ring ? ring + (BL_DEPTH - 1) * PLACE : here - PLACE);
        fetched<BL_DEPTH - 1>();
        __syncwarp();
        float* const mine = here + tig * s.E;  // the token's row; then that of its gradient
        f2 x[N2];
        load_row<LPT, VEC>(mine, there, s.E, lig, x);
        here = here == ring + (BL_DEPTH - 1) * PLACE ? ring : here + PLACE;
        __syncwarp();
        if (there && (seq == -2 || t >= seq_end)) {
            seq = starts.find(s, t);
            seq_end = seq < 0 ? starts(s, 0) : seq < s.S ? starts(s, seq + 1) : s.T;
            seq_live = seq >= 0 && seq < s.S;
#pragma unroll
            for (int i = 0; i < N2; ++i) {
                float v[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int c = column<LPT, VEC>(lig, 2 * i + k);
                    v[k] = seq_live && c < s.E ? wb * slopes[(size_t)seq * s.E + c] : 0.f;
                }
                a[i] = pair(v[0], v[1]);
            }
        }
        exponentials(x, m);
        f2 dots = mul_(x[0], a[0]);
#pragma unroll
        for (int i = 1; i < N2; ++i) dots = fma_(x[i], a[i], dots);
        float dot = total(dots), gd = g0 * d0;
        if (gates) {
            for (int j = LPT; lig + j < s.k; j += LPT)
                if (there) gd = fmaf(gates[at + j], dgates[at + j], gd);
        }
        group_sums<LPT>(dot, gd, lane);
        live = live && seq_live && inv != 0.f;
        // p (a - sum p a + z's part): exp(l - m) times inv (a + c)
        const float c = wz * lse - dot * inv;
        const f2 vi = both<f2>(inv), vc = both<f2>(c * inv);
#pragma unroll
        for (int i = 0; i < N2; ++i) x[i] = mul_(x[i], fma_(a[i], vi, vc));
        if (!live) {
#pragma unroll
            for (int i = 0; i < N2; ++i) x[i] = both<f2>(0.f);
        }
        if (gates) {
            // through shared memory, where a pair's value finds its expert's place; pairs of one token that name the
            // same expert go one after another
            if (VEC) {
#pragma unroll
                for (int q = 0; q < NV / 4; ++q)
                    if (column<LPT, VEC>(lig, 4 * q) < s.E)
                        *reinterpret_cast<ulonglong2*>(mine + column<LPT, VEC>(lig, 4 * q)) = make_ulonglong2(x[2 * q], x[2 * q + 1]);
            } else {
#pragma unroll
                for (int i = 0; i < N2; ++i) {
                    const float2 v = split(x[i]);
                    if (column<LPT, VEC>(lig, 2 * i) < s.E) mine[column<LPT, VEC>(lig, 2 * i)] = v.x;
                    if (column<LPT, VEC>(lig, 2 * i + 1) < s.E) mine[column<LPT, VEC>(lig, 2 * i + 1)] = v.y;
                }
            }
            __syncwarp();
            for (int j0 = 0; j0 < s.k; j0 += LPT) {
                const bool own = live && j0 + lig < s.k;
                const int e = j0 == 0 ? e0 : own ? idx[at + j0] : -1;
                const float v = j0 == 0 ? g0 * (d0 - gd) : own ? gates[at + j0] * (dgates[at + j0] - gd) : 0.f;
                const bool good = own && (unsigned)e < (unsigned)s.E;
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
            if (VEC) {
#pragma unroll
                for (int q = 0; q < NV / 4; ++q) {
                    if (column<LPT, VEC>(lig, 4 * q) >= s.E) continue;
                    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(mine + column<LPT, VEC>(lig, 4 * q));
                    x[2 * q] = v.x;
                    x[2 * q + 1] = v.y;
                }
            } else {
#pragma unroll
                for (int i = 0; i < N2; ++i) {
                    const int c = column<LPT, VEC>(lig, 2 * i), d = column<LPT, VEC>(lig, 2 * i + 1);
                    x[i] = pair(c < s.E ? mine[c] : 0.f, d < s.E ? mine[d] : 0.f);
                }
            }
            __syncwarp();
        }
        if (!there) continue;
        float* const out = dlogits + (size_t)t * s.E;
        if (VEC) {
#pragma unroll
            for (int q = 0; q < NV / 4; ++q) {
                const int c = (q * LPT + lig) * 4;
                if (c < s.E) *reinterpret_cast<ulonglong2*>(out + c) = make_ulonglong2(x[2 * q], x[2 * q + 1]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N2; ++i) {
                const float2 v = split(x[i]);
                const int c = 2 * i * LPT + lig;
                if (c < s.E) out[c] = v.x;
                if (c + LPT < s.E) out[c + LPT] = v.y;
            }
        }
    }
    fetched<0>();
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

// Lanes of a token: with eight logits each, as few as hold a row; with more than 128 experts 16 lanes of sixteen: a warp
// that has one token only spends most of its instructions on what a token costs whatever its row's length
// (131072 tokens of 256 experts in 67 sequences, both passes: 91 us instead of 112).
int lanes_of(int E) {
    int l = 1;
    while (l * 8 < E && l < 16) l *= 2;
    return l;
}
int values_of(int E) { return E > 128 ? 16 : 8; }
int ctas_of(const moe_balance_config& c, int threads, int most) {
    const int pass = threads / lanes_of(c.E);  // tokens that a CTA has in its registers at once
    const int n = (c.T + pass - 1) / pass;
    return n < 1 ? 1 : n < most ? n : most;
}
// Forward: as many CTAs as sequences at least, as each ends with barriers and a row of sums, one after another.
int forward_ctas(const moe_balance_config& c, int threads, int most) {
    const int n = ctas_of(c, threads, most), m = c.seqs < c.T ? c.seqs : c.T;
    return n >= m ? n : m < most ? m : most;
}
int most_ctas(const DeviceInfo& di, int threads) {
    const int n = di.sms * (threads < BL_THREADS ? 3 : 1);
    return n < BL_MAX_CTAS ? n : BL_MAX_CTAS;
}
// Large CTAs leave few rows of sums behind (both passes over 16384 tokens of 64 experts: 15.1 us instead of 16.4, over 131072
// 38.2 instead of 40.4). Where they would not all have work, or several sequences would end in one of them, small ones are
// faster (16384 tokens of 64 experts in 300 sequences: 25.5 us instead of 30.5; 2000 in 100: 18.2 instead of 19.7). With 256
// experts the two are close, and small ones ahead where there are many sequences (131072 tokens: 83.5 us with large and 84.4
// with small ones in one sequence, 90.7 and 88.6 in 67); of few tokens and experts large ones are a little (4096 of 8,
// forward: 6.3 us, 6.7 with small ones).
int threads_of(const moe_balance_config& c, int sms) {
    const int pass = BL_THREADS / lanes_of(c.E);
    return c.T / pass >= sms / 2 && c.T / c.seqs >= pass ? BL_THREADS : 256;
}

BlShape shape_of(const moe_balance_config& c, const int32_t* offsets, const uint8_t* mask, int ctas) {
    BlShape s;
    s.T = c.T, s.E = c.E, s.k = c.topk, s.S = c.seqs;
    s.chunk = c.T ? (c.T + ctas - 1) / ctas : 1;
    s.offsets = offsets;
    s.mask = mask;
    return s;
}

size_t ring_bytes(int threads, int E) { return (size_t)threads / 32 * BL_DEPTH * 32 * values_of(E) * 4; }
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

// f(lanes of a token, a lane's values, whole vectors?) for the config.
template <typename F>
cudaError_t dispatch(int E, bool vec, F f) {
    auto on = [&](auto lpt, auto nv) { return vec ? f(lpt, nv, std::true_type()) : f(lpt, nv, std::false_type()); };
    if (values_of(E) == 16) return on(Int<16>(), Int<16>());
    switch (lanes_of(E)) {
        case 1: return on(Int<1>(), Int<8>());
        case 2: return on(Int<2>(), Int<8>());
        case 4: return on(Int<4>(), Int<8>());
        case 8: return on(Int<8>(), Int<8>());
        default: return on(Int<16>(), Int<8>());
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
    *bytes = space_bytes(*c, forward_ctas(*c, 256, BL_MAX_CTAS));
    return MOE_OK;
}

MOE_API int moe_balance_saved_size(const moe_balance_config* c, size_t* bytes) {
    clear_error();
    const int rc = check(c);
    if (rc) return rc;
    if (!bytes) return fail(MOE_ERR_ARG, "bytes is NULL");
    *bytes = 4 * (kept_at(c->seqs, c->E) + 3 * (size_t)c->T);
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
    const int threads = threads_of(*c, di.sms), ctas = forward_ctas(*c, threads, most_ctas(di, threads));
    const size_t need = space_bytes(*c, ctas);
    if (ws_bytes < need) return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
    const BlShape s = shape_of(*c, offsets, mask, ctas);
    const BlSpace w = space_of(*c, ws);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = dispatch(c->E, c->E % 4 == 0 && aligned(logits, 16), [&](auto lpt, auto nv, auto vec) {
        constexpr auto kernel = &balance_kernel<decltype(lpt)::value, decltype(nv)::value, decltype(vec)::value>;
        const cudaError_t e0 = allow_smem<kernel>(ring_bytes(BL_THREADS, c->E));
        if (e0 != cudaSuccess) return e0;
        return launch_k(kernel, dim3(ctas), dim3(threads), ring_bytes(threads, c->E), st, true,
                        s, logits, idx, lse, saved ? reinterpret_cast<BlKept*>(static_cast<float*>(saved) + kept_at(c->seqs, c->E)) : nullptr, w);
    });
    if (e != cudaSuccess) return cuda_fail(e, "balance loss launch");
    BlEnd f;
    f.blocks = (int)blocks_of(c->E);
    f.wb = c->balance, f.wz = c->z;
    f.loss = loss, f.counts = counts, f.saved = static_cast<float*>(saved);
    // as many warps on a job as it has rows on average, up to a CTA's
    f.splits = 1;
    while (f.splits < BL_END_WARPS && f.splits < (ctas + c->seqs - 1) / c->seqs) f.splits *= 2;
    const int jobs = c->seqs * f.blocks, warps = jobs <= BL_END_WARPS / f.splits ? jobs * f.splits : f.splits < 8 ? 8 : f.splits, per = warps / f.splits, n = (jobs + per - 1) / per;
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
    const uintptr_t in = reinterpret_cast<uintptr_t>(logits), to = reinterpret_cast<uintptr_t>(dlogits);
    const size_t bytes = 4 * (size_t)c->T * c->E;
    if (in != to && in < to + bytes && to < in + bytes) return fail(MOE_ERR_ARG, "dlogits shares memory with part of logits");
    DeviceInfo di;
    if ((rc = check_device(&di))) return rc;
    const int ctas = ctas_of(*c, BL_BACK_THREADS, BL_BACK_CTAS * di.sms);
    const BlShape s = shape_of(*c, offsets, mask, ctas);
    const bool vec = c->E % 4 == 0 && aligned(logits, 16) && aligned(dlogits, 16);
    const cudaError_t e = dispatch(c->E, vec, [&](auto lpt, auto nv, auto v) {
        constexpr auto kernel = &balance_backward_kernel<decltype(lpt)::value, decltype(nv)::value, decltype(v)::value>;
        const cudaError_t e0 = allow_smem<kernel>(ring_bytes(BL_BACK_THREADS, c->E));
        if (e0 != cudaSuccess) return e0;
        return launch_k(kernel, dim3(ctas), dim3(BL_BACK_THREADS), ring_bytes(BL_BACK_THREADS, c->E),
                        static_cast<cudaStream_t>(stream), true, s, logits, idx, static_cast<const float*>(saved), gates,
                        dgates, dloss, dlogits);
    });
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "balance loss backward launch");
}

}  // extern "C"
