// Dense gated feed-forward block: forward and backward pass.
//
//   g = x W1^T, u = x W3^T, h = silu(g) * u, y = h W2^T
//   dh = dy W2, s = 1 / (1 + exp(-g)), dg = dh u s (1 + g (1 - s)), du = dh g s
//   dx = dg W1 + du W3, dW1 = dg^T x, dW3 = du^T x, dW2 = dy^T h
//
// Two kernels run the products. dense_kernel is a persistent tcgen05 GEMM on CTA pairs (UMMA 256 x 256 x 16,
// cta_group::2, fp32 accumulators in TMEM, operands by TMA through a seven-stage ring) over a list of
// products. flex_kernel is for few tokens or few tiles: 128 features by 16 to 128 tokens a CTA, the k-blocks
// split over a cluster. An estimate of both, fitted to 15,400 measured launches, says which one a product
// takes (ff_choose). Both read an operand K-major or MN-major, so no transposed copy is ever written: dh, dx
// read the weights and dW1, dW3, dW2 read both operands along their rows.
//   launch 1 (forward)   g and u side by side in one accumulator; epilogue: h, and g, u in fp32
//   launch 2 (forward)   y
//   launch 3 (backward)  dh; epilogue: dg, du from the kept g, u
//   launch 4 (backward)  dx (one sum over dg W1 and du W3), dW1, dW3, dW2 as one list of tiles; for few
//                        tokens dx on flex_kernel and the weight gradients beside it
// With many tokens the block is bound by the tensor cores (18 T d ffn flops against 2 (4 T d + 6 d ffn)
// bytes of tensors), with few by HBM (the weights) or, for a single token of a small block, by the two
// launches that follow one another. Measured (d, ffn; shares of a measured copy's and product's rates):
//   forward, 4096 tokens (4096, 14336)      849 us in a long run under the power limit, 1.70 PF (99 % of the
//                                           sustained rate), 741-764 us in a short one
//   forward, 37 tokens (4096, 14336)        66 us, 5.3 TB/s (78 %)
//   forward, 1 token (2048, 1408)           10 us, two launches of 3.5 to 5 us
//   both passes, 8192 tokens (2048, 5632)   1142 us, 1.49 PF (79 %; 87 % of the sustained rate)
// g and u are kept in fp32: rounding them would round dg and du twice, and computing them again costs 4 T d ffn
// flops where keeping them costs 16 T ffn bytes of traffic. At d = 2048 and the measured rates that is 199 us
// against 109 us (8192 tokens, ffn 5632). The traffic is not hidden: launches 1 and 3 then keep the tensor pipes
// 72 % and 54 % busy, where launch 4 reaches 88 %, which is about 105 us of the pass.
// h, dg and du are rounded to bf16 because they are operands of the next product.
#include <atomic>

#include "host_internal.h"
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int FT_M = 256, FT_N = 256;   // tile of a CTA pair
constexpr int FF_STAGES = 7;
constexpr int FF_HALF = 128 * BK * 2;   // one CTA's half of an operand's stage: 16 KB
constexpr int FF_STAGE = 2 * FF_HALF;
constexpr int FF_MISC = 1024;
constexpr int FF_WARPS = 8;             // epilogue warps: two for each 32 rows, half of the columns each
constexpr int FF_THREADS = 64 + 32 * FF_WARPS;
constexpr int FF_SMEM = FF_STAGES * FF_STAGE + FF_MISC + 1024;
static_assert(FF_SMEM <= 227 * 1024, "dense GEMM shared memory");
constexpr int FF_PROBLEMS = 4;
// Parts of cut tiles in a launch, and words of the status area: [0] status, [1] detail, [128...] arrivals.
constexpr int FF_MAX_CUT = 160, FF_ARRIVED = 128;
static_assert((FF_ARRIVED + FF_MAX_CUT / 2 * 2 * FF_WARPS) * 4 <= MOE_FFN_STATUS_BYTES, "arrival counts");

enum FfMode : int { FF_PLAIN = 0, FF_SWIGLU = 1, FF_DACT = 2 };

template <int N>
struct FxInt {
    static constexpr int value = N;
};

// One product out[M, N] = sum_k A B of a launch.
struct FfProblem {
    CUtensorMap a[2], b[2];          // the sum runs over operand pair 0, then pair 1 (dx)
    __nv_bfloat16* out[2];           // [M][N]
    int M, N, kb0, kb;               // k-blocks of 64: of pair 0, of both
    int tiles_m, tiles_n;
    int a_mn, b_mn;                  // operand stored along its M / N dimension
    // Units of work: the first `whole` tiles, then each of the others in `parts` parts of its k-blocks.
    int unit0, whole, parts, cut0, slot0;  // first unit, cut tile and part of a cut tile in the launch
    int cut() const { return tiles_m * tiles_n - whole; }
    int units() const { return whole + cut() * parts; }
};
struct FfLaunch {
    FfProblem p[FF_PROBLEMS];
    int count, units;
    int first, extra;        // see ff_unit
    float* partial;          // partial sums of cut tiles, and
    uint32_t* arrived;       // counts of the parts done, one for each epilogue warp of a cut tile (zero between calls)
    float* gu;         // kept g and u (FF_SWIGLU writes, may be null; FF_DACT reads)
    int gu_cols;       // 32-column blocks of a row of it
    int32_t* status;   // [2] first error of the calls on a workspace, and where
    unsigned long long timeout_ns;
    // The launch before this one is not read or overwritten, and all of its CTAs had waited for what came
    // before it when they let this one begin: this launch starts beside it, and waits for it at its
    // end only, so that what follows this launch follows both.
    int beside;
    uint32_t stall;    // test hook, one bit for each rank: stop loading in the middle of the first tile
};

struct FfSmem {
    uint8_t* stages;
    uint64_t *full, *empty, *acc_full, *acc_empty, *drain;
    uint32_t *tmem_base, *peer_base;
    volatile uint32_t* peer_k;
    volatile int* abort;
};
__device__ __forceinline__ FfSmem ff_carve(uint8_t* raw) {
    FfSmem s;
    const uint32_t a = smem_u32(raw);
    uint8_t* base = raw + (((a + 1023u) & ~1023u) - a);
    s.stages = base;
    s.full = reinterpret_cast<uint64_t*>(base + FF_STAGES * FF_STAGE);
    s.empty = s.full + FF_STAGES;
    s.acc_full = s.empty + FF_STAGES;
    s.acc_empty = s.acc_full + 2;
    s.drain = s.acc_empty + 2;
    s.tmem_base = reinterpret_cast<uint32_t*>(s.drain + 1);
    s.peer_base = s.tmem_base + 1;
    s.peer_k = s.peer_base + 1;
    s.abort = reinterpret_cast<volatile int*>(s.tmem_base + 3);
    return s;
}

__device__ __forceinline__ void ff_status(int32_t* status, int detail) {
    if (atomicCAS(&status[0], 0, (int)ST_PIPE_TIMEOUT) == 0) atomicExch(&status[1], detail);
}
__device__ __forceinline__ void ff_abort(const FfSmem& s, uint32_t rank) {
    *s.abort = 1;
    st_cluster_u32(mapa_shared(smem_u32(const_cast<int*>(s.abort)), rank ^ 1u), 1u);
}
// What a CTA waits for before it leaves, products and loads in flight, it waits for this long at least,
// however short the caller's limit on the other waits.
__device__ __forceinline__ unsigned long long ff_hold(unsigned long long tmo) {
    return tmo > 2000000000ull ? tmo : 2000000000ull;
}
// Abort path (rank 0, after both CTAs have stopped issuing): rank 0 armed and loaded `a` k-blocks,
// rank 1 loaded `b`. Bytes that will never come are completed, phases that were never armed are
// armed, then every stage's last phase is waited for: no load is in flight when the CTAs leave.
__device__ __forceinline__ void ff_settle(const FfSmem& s, uint32_t a, uint32_t b, unsigned long long tmo) {
    const uint32_t lo = a < b ? a : b, hi = a < b ? b : a;
    for (uint32_t i = lo; i < hi; ++i) {
        uint64_t* bar = &s.full[i % FF_STAGES];
        if (i < a) mbar_complete_tx(bar, FF_STAGE);
        else mbar_arrive_expect_tx(bar, FF_STAGE);
    }
    int never = 0;
    for (uint32_t i = hi > (uint32_t)FF_STAGES ? hi - FF_STAGES : 0u; i < hi; ++i)
        mbar_wait(&s.full[i % FF_STAGES], (i / FF_STAGES) & 1u, tmo, &never);
}

// Shared-memory descriptor of an operand with the 128-byte swizzle. K-major: rows of 64 k values,
// eight rows 1024 bytes apart. MN-major: blocks of 64 consecutive m (n) by 64 k, a row of 128
// bytes per k, eight k 1024 bytes apart (stride offset), the next 64 m (n) 8 KB on (leading offset).
__device__ __forceinline__ uint64_t ff_sdesc(uint32_t addr, int mn) {
    uint64_t d = sdesc_sw128(addr);
    if (mn) d = (d & ~(uint64_t(0x3FFF) << 16)) | (uint64_t((64 * BK * 2) >> 4) << 16);
    return d;
}
// One operand half (128 rows of M or N from `row`, k-block at `k`) into `dst`; PEER: the odd CTA of a
// pair, whose loads complete on the even CTA's barrier (bar0). How the operands are stored is known at
// compile time here and in the loops below: with run-time branches around the TMA and UMMA issue a
// prompt's products took 10 % longer (930 against 840 us).
template <bool MN, bool PEER>
__device__ __forceinline__ void ff_load(uint8_t* dst, const CUtensorMap* m, uint64_t* bar, uint32_t bar0, int row, int k) {
    if constexpr (!MN) {
        if (PEER) tma_load_2d_pair(dst, m, bar0, k, row);
        else tma_load_2d(dst, m, bar, k, row);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (PEER) tma_load_2d_pair(dst + i * (FF_HALF / 2), m, bar0, row + 64 * i, k);
            else tma_load_2d(dst + i * (FF_HALF / 2), m, bar, row + 64 * i, k);
        }
    }
}
// Place in the ring of stages: stage, phase parity, k-blocks so far.
struct FfRing {
    int st = 0;
    uint32_t ph = 0, done = 0;
    __device__ __forceinline__ void next() {
        ++done;
        if (++st == FF_STAGES) {
            st = 0;
            ph ^= 1u;
        }
    }
};
// TMA thread: k-blocks [from, to) of one operand pair. False if a wait ran out.
template <bool A_MN, bool B_MN, bool PEER>
__device__ __forceinline__ bool ff_produce(const FfSmem& sm, FfRing& r, const CUtensorMap* ma, const CUtensorMap* mb,
                                           int arow, int brow, int from, int to, unsigned long long tmo) {
    for (int kb = from; kb < to; ++kb) {
        if (!mbar_wait(&sm.empty[r.st], r.ph ^ 1u, tmo, sm.abort)) return false;
        uint8_t* a = sm.stages + r.st * FF_STAGE;
        uint64_t* full = &sm.full[r.st];
        uint32_t full0 = 0;
        if (PEER) full0 = mapa_shared(smem_u32(full), 0u);
        else mbar_arrive_expect_tx(full, 2 * FF_STAGE);
        ff_load<A_MN, PEER>(a, ma, full, full0, arow, kb * BK);
        ff_load<B_MN, PEER>(a + FF_HALF, mb, full, full0, brow, kb * BK);
        r.next();
    }
    return true;
}
// UMMA thread (even CTA): `count` k-blocks into the accumulator at dt. False if a wait ran out.
template <bool A_MN, bool B_MN>
__device__ __forceinline__ bool ff_multiply(const FfSmem& sm, FfRing& r, uint32_t dt, int count, unsigned long long tmo) {
    constexpr uint32_t idesc = umma_idesc_bf16(FT_M, FT_N) | ((uint32_t)A_MN << 15) | ((uint32_t)B_MN << 16);
    constexpr uint32_t astep = A_MN ? 128 : 2, bstep = B_MN ? 128 : 2;  // 16 k, in 16 bytes
    for (int kb = 0; kb < count; ++kb) {
        if (!mbar_wait_cluster(&sm.full[r.st], r.ph, tmo, sm.abort)) return false;
        tc_fence_after();
        const uint32_t addr = smem_u32(sm.stages + r.st * FF_STAGE);
        const uint64_t ad = ff_sdesc(addr, A_MN), bd = ff_sdesc(addr + FF_HALF, B_MN);
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk) umma_bf16_pair(dt, ad + astep * kk, bd + bstep * kk, idesc, (kb | kk) != 0);
        umma_commit_pair(&sm.empty[r.st], 0x3);
        r.next();
    }
    return true;
}

// Arrive on a barrier of the pair without ordering this thread's memory operations: the epilogue's signal
// that it has read the accumulator. Its tcgen05 loads have completed (wait::ld) and
// tcgen05.fence::before_thread_sync orders them before the arrive, as fence::after_thread_sync orders the UMMAs
// after the wait for it; a releasing arrive would wait for the stores in flight as well.
__device__ __forceinline__ void ff_arrive_relaxed(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// One unit of work: a tile, or one part of a cut tile (cut: its number among them, -1: none).
// The product's numbers are copied here, into registers: read through the pointer into the launch's
// parameters they would be loaded again for every k-block.
struct FfTile {
    const FfProblem* p;
    int m, n, k0, k1, cut, part, parts;
    int M, N, kb0, a_mn, b_mn;
};
// The i-th unit of a cluster (-1: no more). The first l.first units, which take longer, go round the
// clusters; those that got one less then take l.extra of the others; the rest goes round again, from them on.
__device__ __forceinline__ int ff_unit(const FfLaunch& l, int cluster, int clusters, int i) {
    int u = cluster + i * clusters;
    if (u >= l.first) {
        const int rounds = l.first / clusters, high = l.first - rounds * clusters;
        int c = cluster - high;
        i -= rounds;
        u = l.first;
        if (c < 0) {
            i -= 1;
            c += clusters;
            u += l.extra * (clusters - high) + c + i * clusters;
        } else if (i < l.extra) {
            u += c + i * (clusters - high);
        } else {
            u += l.extra * (clusters - high) + c + (i - l.extra) * clusters;
        }
    }
    return u < l.units ? u : -1;
}
__device__ __forceinline__ FfTile ff_tile(const FfLaunch& l, int unit) {
    int i = 0;
    while (i + 1 < l.count && unit >= l.p[i + 1].unit0) ++i;
    const FfProblem* p = &l.p[i];
    int q = unit - p->unit0, part = 0, cut = -1;
    const int whole = p->whole, parts = p->parts;
    if (q >= whole) {
        const int v = q - whole, c = v / parts;
        part = v - c * parts;
        cut = p->cut0 + c;
        q = whole + c;
    }
    // M tiles in groups of 16, N tiles outer in a group: tiles that run together share operands in L2
    const int per = 16 * p->tiles_n, grp = q / per, first = grp * 16;
    const int rows = min(16, p->tiles_m - first), r = q - grp * per;
    FfTile o{p, first + r % rows, r / rows, 0, p->kb, cut, part, parts, p->M, p->N, p->kb0, p->a_mn, p->b_mn};
    if (cut >= 0) {
        const int kb = o.k1;
        o.k0 = kb * part / parts;
        o.k1 = kb * (part + 1) / parts;
    }
    return o;
}

// 32 registers of each lane into 32 lanes x 32 columns of TMEM, then wait.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
        : "memory");
}

// 32 columns of a lane's row as bf16, straight from registers: whole 32-byte sectors where the rows are so
// aligned (`wide`), else 16 bytes at a time. (Staged in shared memory and stored by TMA, 3376 x 3656 values
// took 15.0 us instead of 10.8 us, most of it the proxy fences.)
__device__ __forceinline__ void ff_store(__nv_bfloat16* to, const uint32_t (&pk)[16], int columns, bool wide) {
    if (wide) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (16 * i < columns)
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + 16 * i), "r"(pk[8 * i]),
                             "r"(pk[8 * i + 1]), "r"(pk[8 * i + 2]), "r"(pk[8 * i + 3]), "r"(pk[8 * i + 4]),
                             "r"(pk[8 * i + 5]), "r"(pk[8 * i + 6]), "r"(pk[8 * i + 7])
                             : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (8 * i < columns)
                *reinterpret_cast<uint4*>(to + 8 * i) = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
    }
}

__device__ __forceinline__ float ff_sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

// Kept g and u of a 32 x 32 block: [8 pieces of 4 columns][32 rows][4] fp32, g then u, so that a
// warp whose lanes hold rows reads and writes 512 contiguous bytes at a time.
__device__ __forceinline__ float4* ff_gu(const FfLaunch& l, int row0, int col0, int which, int lane) {
    const size_t block = (size_t)(row0 >> 5) * l.gu_cols + (col0 >> 5);
    return reinterpret_cast<float4*>(l.gu + (block * 2 + which) * 1024) + lane;
}

// The accumulator's 32-column chunk that is the i-th of an epilogue warp's four (half: its half of the
// columns). FF_SWIGLU: chunks 0-3 hold g, 4-7 u of the same features.
template <int MODE>
__device__ __forceinline__ int ff_chunk(int half, int i) {
    return MODE == FF_SWIGLU ? 2 * half + (i & 1) + (i & 2) * 2 : 4 * half + i;
}
// Partial sums of a cut tile's part, for each epilogue warp of the pair (slab): its four chunks, each
// [8 pieces of 4 columns][32 rows][4] fp32.
__device__ __forceinline__ float4* ff_partial(const FfLaunch& l, const FfTile& t, int part, int slab, int lane) {
    const int slot = t.p->slot0 + (t.cut - t.p->cut0) * t.parts + part;
    return reinterpret_cast<float4*>(l.partial + ((size_t)slot * 16 + slab) * 4096) + lane;
}
// A part of a cut tile: keeps this warp's sums and counts them as done. In the part that comes last,
// all parts' sums are added up in their order, put back into the accumulator, and the warp goes on to
// finish its values (true). Nothing waits for another CTA.
template <int MODE>
__device__ __forceinline__ bool ff_collect(const FfLaunch& l, const FfTile& t, uint32_t tb, int half, int slab, int lane) {
    float4* o = ff_partial(l, t, t.part, slab, lane);
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        uint32_t v[32];
        tmem_ld32(tb + ff_chunk<MODE>(half, i) * 32, v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            __stcg(o + i * 256 + k * 32, make_float4(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]),
                                                     __uint_as_float(v[4 * k + 2]), __uint_as_float(v[4 * k + 3])));
    }
    __threadfence();
    __syncwarp();
    uint32_t before = 0;
    if (lane == 0) {
        uint32_t* count = l.arrived + t.cut * 16 + slab;
        before = atom_acq_rel_gpu_add(count, 1u);
        if (before + 1 == (uint32_t)t.parts) *count = 0;  // for the next launch
    }
    before = __shfl_sync(0xffffffffu, before, 0);
    if (before + 1 != (uint32_t)t.parts) return false;
    __threadfence();
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        uint32_t v[32];
        float4 next[8];  // a part's sums are in flight while the one before is added
        auto load = [&](int q) {
            if (q >= t.parts || q == t.part) return;
            const float4* from = ff_partial(l, t, q, slab, lane) + i * 256;
#pragma unroll
            for (int k = 0; k < 8; ++k) next[k] = __ldcg(from + k * 32);
        };
        load(0);
        tmem_ld32(tb + ff_chunk<MODE>(half, i) * 32, v);
        float sum[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) sum[k] = 0.f;
        for (int q = 0; q < t.parts; ++q) {
            float4 cur[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                cur[k] = q == t.part ? make_float4(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]),
                                                   __uint_as_float(v[4 * k + 2]), __uint_as_float(v[4 * k + 3]))
                                     : next[k];
            load(q + 1);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sum[4 * k] += cur[k].x;
                sum[4 * k + 1] += cur[k].y;
                sum[4 * k + 2] += cur[k].z;
                sum[4 * k + 3] += cur[k].w;
            }
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(sum[k]);
        __syncwarp();
        tmem_st32(tb + ff_chunk<MODE>(half, i) * 32, v);
    }
    return true;
}

// Kept g and u of 16 columns of this warp's rows, fetched ahead of their use.
struct FfKept {
    float4 g[4], u[4];
    // the k-th 16 of a warp's 128 columns
    __device__ __forceinline__ void load(const FfLaunch& l, const FfTile& t, int row0, int half, int k, int lane) {
        const int col0 = t.n * FT_N + half * 128 + (k & ~1) * 16;
        if (row0 >= t.M || k >= 8 || col0 >= t.N) return;
        const float4 *ig = ff_gu(l, row0, col0, 0, lane) + (k & 1) * 128, *iu = ff_gu(l, row0, col0, 1, lane) + (k & 1) * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            g[i] = __ldcs(ig + i * 32);
            u[i] = __ldcs(iu + i * 32);
        }
    }
};

// `release` is called once per tile, when the warp has read its part of the accumulator.
template <int MODE, typename Release>
__device__ __forceinline__ void ff_epilogue(const FfLaunch& l, const FfTile& t, uint32_t tb, int row0,
                                            int half, int slab, int lane, FfKept& next, Release release) {
    if (row0 >= t.M) {
        release();
        return;
    }
    __nv_bfloat16* const out = t.p->out[0] + (size_t)(row0 + lane) * t.N;
    __nv_bfloat16* const out1 = MODE == FF_DACT ? t.p->out[1] + (size_t)(row0 + lane) * t.N : nullptr;
    const bool in = row0 + lane < t.M;
    const bool wide = t.N % 16 == 0 && ((reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(out1)) & 31) == 0;
    if (t.cut >= 0 && !ff_collect<MODE>(l, t, tb, half, slab, lane)) {
        release();
        return;
    }
    if (MODE == FF_SWIGLU) {
#pragma unroll 1
        for (int c = 2 * half; c < 2 * half + 2; ++c) {
            const int col0 = t.n * 128 + c * 32;
            if (col0 >= t.N) break;
            uint32_t g[32], u[32];
            tmem_ld32(tb + c * 32, g);
            tmem_ld32(tb + 128 + c * 32, u);
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float g0 = __uint_as_float(g[2 * i]), g1 = __uint_as_float(g[2 * i + 1]);
                pk[i] = pack_bf16x2(g0 * ff_sigmoid(g0) * __uint_as_float(u[2 * i]),
                                    g1 * ff_sigmoid(g1) * __uint_as_float(u[2 * i + 1]));
            }
            if (l.gu) {
                float4 *og = ff_gu(l, row0, col0, 0, lane), *ou = ff_gu(l, row0, col0, 1, lane);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    og[i * 32] = make_float4(__uint_as_float(g[4 * i]), __uint_as_float(g[4 * i + 1]),
                                             __uint_as_float(g[4 * i + 2]), __uint_as_float(g[4 * i + 3]));
                    ou[i * 32] = make_float4(__uint_as_float(u[4 * i]), __uint_as_float(u[4 * i + 1]),
                                             __uint_as_float(u[4 * i + 2]), __uint_as_float(u[4 * i + 3]));
                }
            }
            if (in) ff_store(out + col0, pk, t.N - col0, wide);
            __syncwarp();
        }
        release();
    } else if (MODE == FF_DACT) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            const int col0 = t.n * FT_N + half * 128 + c * 32;
            if (col0 >= t.N) break;
            uint32_t d[32];
            tmem_ld32(tb + (4 * half + c) * 32, d);
            uint32_t pg[16], pu[16];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const FfKept k = next;
                next.load(l, t, row0, half, 2 * c + h + 1, lane);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float gv[4] = {k.g[i].x, k.g[i].y, k.g[i].z, k.g[i].w};
                    const float uv[4] = {k.u[i].x, k.u[i].y, k.u[i].z, k.u[i].w};
                    float dg[4], du[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float dh = __uint_as_float(d[h * 16 + 4 * i + j]), s = ff_sigmoid(gv[j]);
                        du[j] = dh * (gv[j] * s);
                        dg[j] = dh * uv[j] * (s * (1.0f + gv[j] * (1.0f - s)));
                    }
                    pg[h * 8 + 2 * i] = pack_bf16x2(dg[0], dg[1]);
                    pg[h * 8 + 2 * i + 1] = pack_bf16x2(dg[2], dg[3]);
                    pu[h * 8 + 2 * i] = pack_bf16x2(du[0], du[1]);
                    pu[h * 8 + 2 * i + 1] = pack_bf16x2(du[2], du[3]);
                }
            }
            if (in) {
                ff_store(out + col0, pg, t.N - col0, wide);
                ff_store(out1 + col0, pu, t.N - col0, wide);
            }
            __syncwarp();
        }
        release();
    } else {
        // everything out of the accumulator first, so that the next products may have it while these values
        // are stored
        uint32_t pk[4][16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t v[32];
            tmem_ld32(tb + (4 * half + i) * 32, v);
#pragma unroll
            for (int k = 0; k < 16; ++k) pk[i][k] = pack_bf16x2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]));
        }
        release();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int col0 = t.n * FT_N + (4 * half + i) * 32;
            if (in && col0 < t.N) ff_store(out + col0, pk[i], t.N - col0, wide);
        }
    }
}

// f(FxInt<bit 0: A, bit 1: B stored along M / N>) for the forms that a kernel's products take: the
// forward products (0), dh and dx (2), the weight gradients (3).
template <int MODE, typename F>
__device__ __forceinline__ void ff_forms(int form, F f) {
    if (MODE == FF_SWIGLU) f(FxInt<0>());
    else if (MODE == FF_DACT) f(FxInt<2>());
    else if (form == 0) f(FxInt<0>());
    else if (form == 2) f(FxInt<2>());
    else f(FxInt<3>());
}

// Persistent GEMM on CTA pairs: each cluster takes the units of work that the launch gives it.
// Warp 0: TMA loads (each CTA its 128 rows of A and 128 of B; both CTAs' loads complete on rank 0's
// stage barrier). Warp 1: TMEM, and on rank 0 the UMMAs. Warps 2-9: epilogue of the CTA's 128 rows,
// overlapping the next tile's products through two accumulators. Every wait is bounded; one that
// runs out raises the pair's abort word and the status word, and the loads in flight are settled.
template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(FF_THREADS, 1)
    dense_kernel(const __grid_constant__ FfLaunch l) {
    extern __shared__ uint8_t smem_raw[];
    const FfSmem sm = ff_carve(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
    const unsigned long long tmo = l.timeout_ns;
    if (tid == 0) {
        for (int i = 0; i < FF_STAGES; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.acc_full[i], 1);
            mbar_init(&sm.acc_empty[i], 2 * FF_WARPS);
        }
        mbar_init(sm.drain, 1);
        *sm.abort = 0;
        mbar_fence_init();
    }
    __syncthreads();
    if (warp == 0 && lane < l.count) {
        tma_prefetch_desc(&l.p[lane].a[0]);
        tma_prefetch_desc(&l.p[lane].b[MODE == FF_SWIGLU ? (int)rank : 0]);
    }
    if (warp == 1) {
        tmem_alloc_pair(sm.tmem_base, TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (rank == 1 && tid == 0) st_cluster_u32(mapa_shared(smem_u32(sm.peer_base), 0u), *sm.tmem_base);
    cluster_sync();
    if (!l.beside) griddep_wait();
    griddep_launch();
    const uint32_t tmem = *sm.tmem_base;
    const bool bad = rank == 0 && *sm.peer_base != tmem;
    uint32_t nk = 0;

    if (warp == 0 && lane == 0) {
        FfRing ring;
        bool ok = !bad;
        const bool stall = l.stall >> rank & 1u;
        for (int i = 0, u; ok && (u = ff_unit(l, cluster, clusters, i)) >= 0; ++i) {
            FfTile tr = ff_tile(l, u);
            if (stall) tr.k1 = tr.k0 + (tr.k1 - tr.k0) / 2;
            const int arow = tr.m * FT_M + (int)rank * 128;
            const int brow = MODE == FF_SWIGLU ? tr.n * 128 : tr.n * FT_N + (int)rank * 128;
            auto load = [&](auto form) {
                constexpr bool A_MN = decltype(form)::value & 1, B_MN = (decltype(form)::value & 2) != 0;
                // the first pair of operands, then (dx) the second
                for (int h = 0; ok && h < 2; ++h) {
                    const int from = h ? max(0, tr.k0 - tr.kb0) : tr.k0, to = h ? tr.k1 - tr.kb0 : min(tr.k1, tr.kb0);
                    const CUtensorMap *ma = tr.p->a + h, *mb = tr.p->b + (MODE == FF_SWIGLU ? (int)rank : h);
                    if (rank == 0) ok = ff_produce<A_MN, B_MN, false>(sm, ring, ma, mb, arow, brow, from, to, tmo);
                    else ok = ff_produce<A_MN, B_MN, true>(sm, ring, ma, mb, arow, brow, from, to, tmo);
                }
            };
            ff_forms<MODE>(tr.a_mn | tr.b_mn << 1, load);
            if (stall) break;
        }
        nk = ring.done;
        if (!ok) {
            if (!*sm.abort) ff_status(l.status, 10 + (int)rank);
            ff_abort(sm, rank);
        }
    } else if (warp == 1 && lane == 0) {
        bool ok = !bad;
        if (bad) {
            ff_status(l.status, 9);
            ff_abort(sm, rank);
        }
        if (rank == 0) {
            FfRing ring;
            int b = 0;
            uint32_t aph = 0;
            for (int i = 0, u; ok && (u = ff_unit(l, cluster, clusters, i)) >= 0; ++i) {
                const FfTile tr = ff_tile(l, u);
                if (!mbar_wait_cluster(&sm.acc_empty[b], aph ^ 1u, tmo, sm.abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                ff_forms<MODE>(tr.a_mn | tr.b_mn << 1, [&](auto form) {
                    constexpr bool A_MN = decltype(form)::value & 1, B_MN = (decltype(form)::value & 2) != 0;
                    ok = ff_multiply<A_MN, B_MN>(sm, ring, tmem + (uint32_t)(b * 256), tr.k1 - tr.k0, tmo);
                });
                if (!ok) break;
                umma_commit_pair(&sm.acc_full[b], 0x3);
                b ^= 1;
                if (b == 0) aph ^= 1u;
            }
            umma_commit_pair(sm.drain, 0x3);  // fires when every UMMA issued has completed
        }
        if (!ok) {
            if (!*sm.abort) ff_status(l.status, 12 + (int)rank);
            ff_abort(sm, rank);
        }
        int never = 0;
        if (!mbar_wait(sm.drain, 0, ff_hold(tmo), &never) && !*sm.abort) ff_status(l.status, 14 + (int)rank);
    } else if (warp >= 2) {
        const int q = warp & 3, half = (warp - 2) >> 2;
        const uint32_t acc_empty0 = mapa_shared(smem_u32(sm.acc_empty), 0u);
        int b = 0;
        uint32_t aph = 0;
        for (int i = 0, u; !bad && (u = ff_unit(l, cluster, clusters, i)) >= 0; ++i) {
            const FfTile tr = ff_tile(l, u);
            const int row0 = tr.m * FT_M + (int)rank * 128 + q * 32;
            FfKept kept;
            if (MODE == FF_DACT) kept.load(l, tr, row0, half, 0, lane);
            const bool got = mbar_wait(&sm.acc_full[b], aph, tmo, sm.abort);
            if (!__all_sync(0xffffffffu, got)) {  // the whole warp goes on or none of it
                if (lane == 0) {
                    if (!*sm.abort) ff_status(l.status, 16 + (int)rank);
                    ff_abort(sm, rank);
                }
                break;
            }
            tc_fence_after();
            const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * 256);
            ff_epilogue<MODE>(l, tr, tb, row0, half, (int)rank * FF_WARPS + warp - 2, lane, kept, [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) ff_arrive_relaxed(acc_empty0 + b * 8u);
            });
            b ^= 1;
            if (b == 0) aph ^= 1u;
        }
        __syncwarp();
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync();  // both CTAs: all roles done, all UMMAs complete, every abort word written
    if (*sm.abort) {
        if (tid == 0 && rank == 1) st_cluster_u32(mapa_shared(smem_u32(const_cast<uint32_t*>(sm.peer_k)), 0u), nk);
        cluster_sync();
        if (tid == 0 && rank == 0) ff_settle(sm, nk, *sm.peer_k, ff_hold(tmo));
        cluster_sync();
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem, TMEM_COLS);
    }
    __syncwarp();
    cluster_sync();
    if (l.beside) griddep_wait();
}

// ---- few tokens or few tiles: flex_kernel ----------------------------------------------------------
//
// One CTA computes 128 features by NT tokens (NT a multiple of 16 up to 128) of a product in which the
// features come from a weight matrix: the weights are the UMMA's A operand (128 rows), the tokens its B
// operand (N = NT), so few tokens waste no tensor-core rows and every byte of the weights is read once.
// The k-blocks of a tile are split over a cluster of S CTAs, whose partial sums meet in shared memory:
// CTA r of the cluster adds up and finishes the r-th part of the tokens, in CTA order. That puts
// enough CTAs on the weights to read them at the memory's rate when there are few tiles.
// A launch that follows another of the same call (`early`) starts loading weights before it waits for
// the previous kernel: that kernel does not write them, and whatever came before it had finished when it let
// this launch begin (it waits for its predecessor before it triggers its dependants).
struct FxArgs {
    CUtensorMap a[2], b[2];
    int M, T;             // features, tokens
    int kb0, kb;          // k-blocks of operand pair 0, of both (FF_SWIGLU: a[0] and a[1] side by side)
    int nt, splits, tiles_t;
    int stages, early;
    uint32_t stall;       // test hook: stop loading halfway
    __nv_bfloat16 *out0, *out1;  // [T][M]
    float2* gu;                  // kept g and u, [T][M]
    int32_t* status;
    unsigned long long timeout_ns;
};
constexpr int FX_MAX_STAGES = 8;
constexpr int FX_ROOM = 108 * 1024;  // a CTA's ring: two CTAs fit a SM
constexpr int FX_A = 128 * BK * 2;  // bytes of a stage's 128 weight rows
__host__ __device__ inline int fx_stage_bytes(bool dual, int nt) { return (dual ? 2 : 1) * FX_A + nt * BK * 2; }

// Where a thread's results go: its feature of some token, the next token M values on.
template <int MODE>
struct FxOut {
    __nv_bfloat16 *o0, *o1;
    float2* gu;
    int M;
    __device__ __forceinline__ FxOut(const FxArgs& p, int t, int f) : M(p.M) {
        const size_t at = (size_t)t * p.M + f;
        o0 = p.out0 + at;
        o1 = p.out1 + at;
        gu = p.gu ? p.gu + at : nullptr;
    }
    __device__ __forceinline__ float2 kept(int j) const {
        return MODE == FF_DACT ? gu[(size_t)j * M] : make_float2(0.f, 0.f);
    }
    // Token j on from the first: its value (and, for h, the second product's).
    __device__ __forceinline__ void put(int j, float v, float w, float2 k) const {
        const size_t at = (size_t)j * M;
        if (MODE == FF_SWIGLU) {
            o0[at] = __float2bfloat16_rn(v * ff_sigmoid(v) * w);
            if (gu) gu[at] = make_float2(v, w);
        } else if (MODE == FF_DACT) {
            const float s = ff_sigmoid(k.x);
            o0[at] = __float2bfloat16_rn(v * k.y * (s * (1.0f + k.x * (1.0f - s))));
            o1[at] = __float2bfloat16_rn(v * (k.x * s));
        } else {
            o0[at] = __float2bfloat16_rn(v);
        }
    }
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
// W (2 or 4) consecutive floats into a peer's shared memory / from our own.
template <int W>
__device__ __forceinline__ void st_cluster_vec(uint32_t cluster_addr, const uint32_t* v) {
    if (W == 4)
        asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "r"(v[0]), "r"(v[1]),
                     "r"(v[2]), "r"(v[3])
                     : "memory");
    else
        asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(cluster_addr), "r"(v[0]), "r"(v[1]) : "memory");
}
template <int W>
struct alignas(4 * W) FxVec {
    float v[W];
};

template <int MODE, bool A_MN>
__global__ void __launch_bounds__(GEMM_THREADS, 1) flex_kernel(const __grid_constant__ FxArgs p) {
    constexpr bool DUAL = MODE == FF_SWIGLU;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[FX_MAX_STAGES], empty[FX_MAX_STAGES], done;
    __shared__ uint32_t tmem_base;
    __shared__ volatile int abort_word;
    uint8_t* const ring = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = p.splits, split = S > 1 ? (int)cluster_ctarank() : 0;
    const int tile = (int)blockIdx.x / S, mt = tile / p.tiles_t, tt = tile - mt * p.tiles_t;
    const int f0 = mt * 128, t0 = tt * p.nt;
    const int k0 = (int)((int64_t)p.kb * split / S), nkb = (int)((int64_t)p.kb * (split + 1) / S) - k0;
    const int stage_bytes = fx_stage_bytes(DUAL, p.nt);
    const unsigned long long tmo = p.timeout_ns;
    uint32_t cols = 32;
    while (cols < (uint32_t)(DUAL ? 2 * p.nt : p.nt)) cols *= 2;
    if (tid == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(&done, 1);
        abort_word = 0;
        mbar_fence_init();
    }
    if (warp == 0 && lane == 1) {
        tma_prefetch_desc(&p.a[0]);
        tma_prefetch_desc(&p.b[0]);
        if (DUAL) tma_prefetch_desc(&p.a[1]);
    }
    if (warp == 1) {
        tmem_alloc(&tmem_base, cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            auto pair_of = [&](int kb) { return kb >= p.kb0 ? 1 : 0; };
            auto weights = [&](int kb, int st) {
                const int second = pair_of(kb), k = (kb - (second ? p.kb0 : 0)) * BK;
                uint8_t* a = ring + st * stage_bytes;
                mbar_arrive_expect_tx(&full[st], stage_bytes);
                ff_load<A_MN, false>(a, &p.a[second], &full[st], 0u, f0, k);
                if (DUAL) ff_load<A_MN, false>(a + FX_A, &p.a[1], &full[st], 0u, f0, k);
            };
            auto tokens = [&](int kb, int st) {
                const int second = pair_of(kb), k = (kb - (second ? p.kb0 : 0)) * BK;
                tma_load_2d(ring + st * stage_bytes + (DUAL ? 2 : 1) * FX_A, &p.b[second], &full[st], k, t0);
            };
            const int loads = p.stall ? nkb / 2 : nkb;
            const int head = loads < p.stages ? loads : p.stages;
            if (p.early)
                for (int i = 0; i < head; ++i) weights(k0 + i, i);
            griddep_wait();
            griddep_launch();
            int issued = 0, st = 0;
            uint32_t ph = 0;
            for (; issued < head; ++issued) {
                if (!p.early) weights(k0 + issued, issued);
                tokens(k0 + issued, issued);
            }
            for (; issued < loads; ++issued) {  // stage st is free once its products of round ph are done
                if (!mbar_wait(&empty[st], ph, tmo, &abort_word)) {
                    ok = false;
                    break;
                }
                weights(k0 + issued, st);
                tokens(k0 + issued, st);
                if (++st == p.stages) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            if (!ok) {
                if (!abort_word) ff_status(p.status, 20);
                abort_word = 1;
            }
            // no load is in flight when the CTA leaves: each stage's last phase has completed
            int never = 0;
            for (int i = issued > p.stages ? issued - p.stages : 0; i < issued; ++i)
                if (!mbar_wait(&full[i % p.stages], (uint32_t)(i / p.stages) & 1u, ff_hold(tmo), &never)) ff_status(p.status, 21);
        }
    } else if (warp == 1) {
        griddep_wait();
        griddep_launch();
        if (lane == 0) {
            const uint32_t idesc = umma_idesc_bf16(128, p.nt) | ((uint32_t)A_MN << 15);
            constexpr uint32_t astep = A_MN ? 128 : 2;
            int st = 0;
            uint32_t ph = 0;
            for (int i = 0; i < nkb; ++i) {
                if (!mbar_wait(&full[st], ph, tmo, &abort_word)) {
                    if (!abort_word) ff_status(p.status, 22);
                    abort_word = 1;
                    break;
                }
                tc_fence_after();
                const uint32_t a = smem_u32(ring + st * stage_bytes), b = a + (DUAL ? 2 : 1) * FX_A;
                const uint64_t ad = ff_sdesc(a, A_MN), ud = ff_sdesc(a + FX_A, A_MN), bd = sdesc_sw128(b);
#pragma unroll
                for (int kk = 0; kk < BK / 16; ++kk) {
                    umma_bf16(tmem, ad + astep * kk, bd + 2 * kk, idesc, (i | kk) != 0);
                    if (DUAL) umma_bf16(tmem + p.nt, ud + astep * kk, bd + 2 * kk, idesc, (i | kk) != 0);
                }
                umma_commit(&empty[st]);
                if (++st == p.stages) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            umma_commit(&done);  // fires when every UMMA issued has completed
            int never = 0;
            if (!mbar_wait(&done, 0, ff_hold(tmo), &never)) {
                ff_status(p.status, 23);
                abort_word = 1;
            }
        }
        __syncwarp();
    } else {
        griddep_wait();
        griddep_launch();
    }
    // every role has ended: all loads landed, all products done
    __syncthreads();
    tc_fence_after();
    if (S > 1) cluster_sync();  // in every CTA of the tile: the rings are free for the partial sums
    const int q = warp & 3, f = f0 + q * 32 + lane;
    const bool dead = abort_word != 0;
    const int own = p.nt / S;  // tokens this CTA finishes
    constexpr int VALS = DUAL ? 2 : 1;
    const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16);
    const int here = min(p.nt, p.T - t0);  // tokens of the tile
    if (S == 1) {
        if (warp >= 2) {
            const FxOut<MODE> out(p, t0, f);
            for (int c = 0; c < here; c += 16) {
                uint32_t v[16], w[16];
                __syncwarp();
                tmem_ld16(tb + c, v);
                if (DUAL) tmem_ld16(tb + p.nt + c, w);
                if (dead || f >= p.M) continue;
                auto finish = [&](int n) {
                    float2 k[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (j < n) k[j] = out.kept(c + j);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (j < n) out.put(c + j, __uint_as_float(v[j]), DUAL ? __uint_as_float(w[j]) : 0.f, k[j]);
                };
                if (here - c >= 16) finish(16);
                else finish(here - c);
            }
        }
    } else {
        // partial sums in shared memory: [split][value][own token / W][128 features][W]
        auto exchange = [&](auto width) {
            constexpr int W = decltype(width)::value;
            FxVec<W>* const parts = reinterpret_cast<FxVec<W>*>(ring);
            const int row = q * 32 + lane, groups = own / W;
            if (warp >= 2) {
                for (int c = 0; c < here; c += 16) {
                    uint32_t v[16], w[16];
                    tmem_ld16(tb + c, v);
                    if (DUAL) tmem_ld16(tb + p.nt + c, w);
#pragma unroll
                    for (int j = 0; j < 16; j += W) {
                        const int to = (c + j) / own, i = (c + j - to * own) / W;
                        const uint32_t at = smem_u32(parts + ((split * VALS) * groups + i) * 128 + row);
                        const uint32_t peer = mapa_shared(at, (uint32_t)to);
                        st_cluster_vec<W>(peer, v + j);
                        if (DUAL) st_cluster_vec<W>(peer + groups * 128 * 4 * W, w + j);
                    }
                }
            }
            tc_fence_before();
            cluster_sync();  // every partial sum has arrived
            const int mine = min(own, here - split * own);
            if (warp < 2 || dead || f >= p.M || mine <= 0) return;
            const FxOut<MODE> out(p, t0 + split * own, f);
            for (int i = 0; i * W < mine; ++i) {
                float2 k[W];
                FxVec<W> v{}, w{};
#pragma unroll
                for (int j = 0; j < W; ++j)
                    if (i * W + j < mine) k[j] = out.kept(i * W + j);
                for (int r = 0; r < S; ++r) {
                    const FxVec<W> a = parts[((r * VALS) * groups + i) * 128 + row];
#pragma unroll
                    for (int j = 0; j < W; ++j) v.v[j] += a.v[j];
                    if (DUAL) {
                        const FxVec<W> b = parts[((r * VALS + 1) * groups + i) * 128 + row];
#pragma unroll
                        for (int j = 0; j < W; ++j) w.v[j] += b.v[j];
                    }
                }
#pragma unroll
                for (int j = 0; j < W; ++j)
                    if (i * W + j < mine) out.put(i * W + j, v.v[j], w.v[j], k[j]);
            }
        };
        if (own % 4 == 0) exchange(FxInt<4>());
        else exchange(FxInt<2>());
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, cols);
    }
}

// ---- host side -----------------------------------------------------------------------------------

struct FfLayout {
    size_t T, d, F;
    size_t h, dg, du, partial, ws_bytes;  // workspace: status words, then h (or dg), du, partial sums
    size_t saved_h, saved_gu, saved_bytes;
    int gu_cols;
    unsigned long long timeout_ns;
    uint32_t flags;
};

int ff_layout(const moe_ffn_config* c, FfLayout* o) {
    if (!c) return fail(MOE_ERR_ARG, "config is NULL");
    if (c->T < 0 || c->T >= (1 << 24)) return fail(MOE_ERR_ARG, "T=%d must be in [0, 2^24)", c->T);
    if (c->d <= 0 || c->d % 8 || c->d >= (1 << 20))
        return fail(MOE_ERR_ARG, "d=%d must be a positive multiple of 8 below 2^20", c->d);
    if (c->ffn <= 0 || c->ffn % 8 || c->ffn >= (1 << 20))
        return fail(MOE_ERR_ARG, "ffn=%d must be a positive multiple of 8 below 2^20", c->ffn);
    if (c->flags & ~(MOE_FFN_TEST_STALL0 | MOE_FFN_TEST_STALL1)) return fail(MOE_ERR_ARG, "flags=%#x is not known", c->flags);
    for (int i = 0; i < 3; ++i)
        if (c->reserved[i]) return fail(MOE_ERR_ARG, "reserved fields must be zero");
    FfLayout L;
    L.T = c->T;
    L.d = c->d;
    L.F = c->ffn;
    const size_t hidden = align_up(L.T * L.F * 2, 1024);
    L.h = L.dg = MOE_FFN_STATUS_BYTES;
    L.du = L.dg + hidden;
    L.partial = L.du + hidden;
    // room for the parts of cut tiles: at most FF_MAX_CUT, and no more than 8 parts of every tile there is
    auto tiles = [](size_t m, size_t n) { return (m + FT_M - 1) / FT_M * ((n + FT_N - 1) / FT_N); };
    size_t parts = 8 * (tiles(L.T, 2 * L.F) + tiles(L.T, L.d) + 3 * tiles(L.F, L.d));
    if (parts > FF_MAX_CUT) parts = FF_MAX_CUT;
    L.ws_bytes = L.partial + parts * FT_M * FT_N * 4;
    L.gu_cols = (int)((L.F + 31) / 32);
    L.saved_h = 0;
    L.saved_gu = hidden;
    L.saved_bytes = hidden + (L.T + 31) / 32 * L.gu_cols * 8192;  // at least T F pairs, the flex layout
    L.flags = c->flags;
    L.timeout_ns = (unsigned long long)(c->timeout_us ? c->timeout_us : 2000000u) * 1000ull;
    *o = L;
    return MOE_OK;
}

// bf16 matrix [rows][inner], boxes of 64 inner values by `box` rows with the 128-byte swizzle.
// Out-of-bounds elements read as zero.
int ff_map(CUtensorMap* m, const void* ptr, uint64_t rows, uint64_t inner, uint32_t box) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint64_t dims[2] = {inner, rows}, strides[1] = {inner * 2};
    const cuuint32_t bx[2] = {(cuuint32_t)BK, box}, es[2] = {1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, bx, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MOE_OK : fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed: %d", (int)r);
}

// Operand [mn, k] (K-major) or, with mn set, stored as [k, mn]; its TMA map.
int ff_operand(CUtensorMap* m, const void* ptr, uint64_t mn, uint64_t k, int along_mn) {
    return along_mn ? ff_map(m, ptr, k, mn, BK) : ff_map(m, ptr, mn, k, 128);
}

struct FfList {
    FfLaunch l;
    int rc = MOE_OK;
    FfList() {  // the products' maps are written as they are added, the others not at all
        l.count = l.units = l.first = l.extra = l.beside = 0;
        l.gu = nullptr;
        l.gu_cols = 0;
    }
    // Adds out[M, N] = A[M, K] B[N, K]^T; a2, b2: a second pair of operands of the same shapes.
    FfProblem& add(const void* a, int a_mn, const void* b, int b_mn, void* out, size_t M, size_t N, size_t K,
                   const void* a2 = nullptr, const void* b2 = nullptr) {
        FfProblem& p = l.p[l.count++];
        p.M = (int)M;
        p.N = (int)N;
        p.kb0 = (int)((K + BK - 1) / BK);
        p.kb = a2 ? 2 * p.kb0 : p.kb0;
        p.a_mn = a_mn;
        p.b_mn = b_mn;
        p.tiles_m = (int)((M + FT_M - 1) / FT_M);
        p.tiles_n = (int)((N + FT_N - 1) / FT_N);
        p.whole = p.tiles_m * p.tiles_n;
        p.parts = 1;
        try_(ff_operand(&p.a[0], a, M, K, a_mn));
        try_(ff_operand(&p.b[0], b, N, K, b_mn));
        if (a2) {
            try_(ff_operand(&p.a[1], a2, M, K, a_mn));
            try_(ff_operand(&p.b[1], b2, N, K, b_mn));
        }
        p.out[0] = p.out[1] = static_cast<__nv_bfloat16*>(out);
        return p;
    }
    void try_(int r) {
        if (rc == MOE_OK) rc = r;
    }
};

// Kinds of products, by their epilogue: plain; h; h with g and u kept; the hidden gradients.
enum FfKind : int { FK_PLAIN = 0, FK_H = 1, FK_H_KEPT = 2, FK_ACT = 3 };

// Times in microseconds that the choices below go by, fitted to 15,400 measured launches: 1017 products of 360 to
// 14336 features, 1 to 4096 tokens and 216 to 14336 k, of every kind, with up to 29 plans each. The plan that these
// numbers choose took 1.03 times the time of the best one measured on average, 1.47 times at worst.
constexpr float US_HBM = 6.3e6f;                            // bytes a microsecond from memory
constexpr float US_DENSE = 4.9f, US_DENSE_KB = 0.287f;      // a launch; a k-block of a 256 x 256 tile
constexpr float US_DENSE_WAVE = 1.9f;                       // a wave beside its k-blocks or epilogue
constexpr float US_DENSE_EPI[4] = {1.5f, 0.6f, 2.9f, 9.3f};  // a tile's epilogue, by kind
constexpr float US_CUT_ROUND = 6.3f, US_CUT_PART = 1.1f;    // a round of parts; adding up each further part
constexpr float US_APART = 3.5f;                            // dx in a launch of its own, the next one beside it
constexpr float US_FLEX = 1.45f, US_FLEX_CTA = 1.09f;       // a launch; a CTA beside its k-blocks
constexpr float US_FLEX_BYTES = 150.9e3f;                   // bytes a microsecond into a SM
constexpr float US_FLEX_LATENCY = 1.15f;                    // of a load, shared by the stages in flight
constexpr float US_FLEX_CYCLES = 1.45f / 1.9e3f;            // a cycle of the tensor cores
constexpr float US_FLEX_TOKEN[4] = {0.0015f, 0.0143f, 0.0259f, 0.0325f};  // a token's values, by kind
constexpr float US_FLEX_SPLIT = 0.55f, US_FLEX_EXCHANGE = 0.0236f;  // a cluster; a token's partial sums
constexpr float US_FLEX_TWO = 1.57f, US_FLEX_MORE = 0.86f;  // two CTAs' fixed part on one SM; each CTA beyond

// Tiles come in waves of one a cluster. The tiles of an incomplete last wave are cut along k into as many
// parts as finish soonest.
struct FfCut {
    int full, parts;
    float us;  // of the whole launch
};
FfCut ff_cut(int tiles, int kb, int clusters, int kind = FK_PLAIN) {
    const int full = tiles / clusters, rest = tiles - full * clusters;
    const float work = kb * US_DENSE_KB, epi = US_DENSE_EPI[kind];
    const float before = US_DENSE + full * ((work > epi ? work : epi) + US_DENSE_WAVE) + epi;
    FfCut best{tiles, 1, before + (rest ? work : 0.0f)};
    if (!rest || rest > FF_MAX_CUT / 2) return best;
    for (int parts = 2; parts <= 8 && rest * parts <= FF_MAX_CUT && parts * 4 <= kb; ++parts) {
        const int rounds = (rest * parts + clusters - 1) / clusters;
        const float us = before + rounds * ((kb + parts - 1) / parts * US_DENSE_KB + US_CUT_ROUND) + US_CUT_PART * (parts - 1);
        if (us < best.us) best = FfCut{full * clusters, parts, us};
    }
    return best;
}

// Co-resident CTA pairs of a kernel on the current device (cached per device).
template <int MODE>
cudaError_t ff_clusters(int* out) {
    const void* fn = reinterpret_cast<const void*>(&dense_kernel<MODE>);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    static std::atomic<int> cache[64];
    if ((*out = cache[dev].load(std::memory_order_relaxed)) == 0) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, FF_SMEM);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t q = {};
        q.gridDim = dim3(2, 1, 1);
        q.blockDim = dim3(FF_THREADS, 1, 1);
        q.dynamicSmemBytes = FF_SMEM;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, fn, &q);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorInvalidConfiguration;
        cache[dev].store(n, std::memory_order_relaxed);
        *out = n;
    }
    return cudaSuccess;
}

// Numbers the units. Where all tiles take alike, those of the last incomplete wave are cut before.
void ff_lay_out(FfLaunch& l, int clusters) {
    if (!l.first) {
        int tiles = 0;
        for (int i = 0; i < l.count; ++i) tiles += l.p[i].whole;
        const FfCut cut = ff_cut(tiles, l.p[0].kb, clusters);
        for (int i = l.count - 1, rest = cut.parts > 1 ? tiles - cut.full : 0; rest; --i) {
            FfProblem& p = l.p[i];
            const int n = rest < p.whole ? rest : p.whole;
            p.whole -= n;
            p.parts = cut.parts;
            rest -= n;
        }
    }
    int cuts = 0, slots = 0;
    l.units = 0;
    for (int i = 0; i < l.count; ++i) {
        FfProblem& p = l.p[i];
        p.unit0 = l.units;
        p.cut0 = cuts;
        p.slot0 = slots;
        l.units += p.units();
        cuts += p.cut();
        slots += p.cut() * p.parts;
    }
}

template <int MODE>
int ff_run(FfList& list, const FfLayout& L, void* ws, cudaStream_t st, const char* what) {
    if (list.rc) return list.rc;
    FfLaunch& l = list.l;
    l.status = static_cast<int32_t*>(ws);
    l.timeout_ns = L.timeout_ns;
    l.stall = L.flags;  // the flags' bits are the ranks'
    l.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + L.partial);
    l.arrived = static_cast<uint32_t*>(ws) + FF_ARRIVED;
    int clusters = 0;
    cudaError_t e = ff_clusters<MODE>(&clusters);
    if (e == cudaSuccess) {
        ff_lay_out(l, clusters);
        const int n = l.units < clusters ? l.units : clusters;
        e = launch_k(dense_kernel<MODE>, dim3(2 * n), dim3(FF_THREADS), FF_SMEM, st, true, list.l);
    }
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, what);
}

// How a product runs: on dense_kernel (nt = 0) or on flex_kernel with these numbers.
struct FxPlan {
    int nt, splits, stages;
    float us;  // the estimate it was chosen by
};

// The quickest flex_kernel plan for a product out[T][M] over kb k-blocks. A k-block costs a CTA the
// tensor cores' time (VALS x 4 UMMAs of max(nt / 2, 32 + nt / 4) cycles: their own, or the shared
// memory's that feeds them 128 x 16 weights and nt x 16 tokens), its bytes' way into the SM, or its share
// of a load's latency; two CTAs on a SM share the first two. Clusters of 4 and 8 do not fill every SM.
FxPlan ff_choose_flex(int M, int T, int kb, int kind, int sms) {
    FxPlan best{0, 1, 0, 1e30f};
    const bool dual = kind == FK_H || kind == FK_H_KEPT;
    const int vals = dual ? 2 : 1;
    const float hbm = (float)M * kb * BK * 2 * vals / US_HBM + 1.7f;
    for (int nt = 16; nt <= 128; nt += nt < 64 ? 16 : 32) {
        if (nt > 16 && nt - (nt <= 64 ? 16 : 32) >= T) break;  // a narrower tile holds every token
        const int stage = fx_stage_bytes(dual, nt), tiles = ((M + 127) / 128) * ((T + nt - 1) / nt);
        const int stages = FX_ROOM / stage < FX_MAX_STAGES ? FX_ROOM / stage : FX_MAX_STAGES;
        const float cycles = US_FLEX_CYCLES * vals * 4 * (nt / 2 > 32 + nt / 4 ? nt / 2 : 32 + nt / 4);
        const float bytes = stage / US_FLEX_BYTES, work = cycles > bytes ? cycles : bytes, wait = US_FLEX_LATENCY / stages;
        const float one = work > wait ? work : wait, two = 2 * work > wait ? 2 * work : wait;
        for (int S = 1; S <= 8; S *= 2) {
            if (S > kb || nt % S || (S > 1 && vals * nt * 512 > stages * stage)) continue;
            const int slots = S == 8 ? sms * 85 / 100 : S == 4 ? sms * 93 / 100 : sms;
            const int load = (tiles * S + slots - 1) / slots, mine = (kb + S - 1) / S;
            const float fixed = US_FLEX_CTA + US_FLEX_TOKEN[kind] * nt / S +
                                (S > 1 ? US_FLEX_SPLIT + US_FLEX_EXCHANGE * nt * vals : 0.0f);
            float us = load / 2 * (mine * two + fixed * US_FLEX_TWO) + load % 2 * (mine * one + fixed) +
                       (load > 2 ? US_FLEX_MORE * (load - 2) : 0.0f);
            us = US_FLEX + (us > hbm ? us : hbm);
            if (us < best.us) best = FxPlan{nt, S, stages, us};
        }
    }
    return best;
}
// dense_kernel's estimate.
FxPlan ff_dense(int M, int T, int kb, int kind, int sms) {
    const bool dual = kind == FK_H || kind == FK_H_KEPT;
    const int tiles = ((T + FT_M - 1) / FT_M) * ((M + (dual ? 127 : FT_N - 1)) / (dual ? 128 : FT_N));
    const float hbm = (float)M * kb * BK * 2 * (dual ? 2 : 1) / US_HBM + 6.7f, us = ff_cut(tiles, kb, sms / 2, kind).us;
    return FxPlan{0, 1, 0, us > hbm ? us : hbm};
}
// The quicker of the two.
FxPlan ff_choose(int M, int T, int kb, int kind, int sms) {
    const FxPlan flex = ff_choose_flex(M, T, kb, kind, sms), dense = ff_dense(M, T, kb, kind, sms);
    return flex.us < dense.us ? flex : dense;
}

// Once per device: the kernel may take FX_ROOM of shared memory.
template <int MODE, bool A_MN>
cudaError_t fx_prepare() {
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&flex_kernel<MODE, A_MN>),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, FX_ROOM + 1024);
    if (e == cudaSuccess) done[dev].store(true, std::memory_order_relaxed);
    return e;
}

template <int MODE, bool A_MN>
int fx_run(FxArgs& p, const FxPlan& plan, const FfLayout& L, void* ws, cudaStream_t st, const char* what) {
    p.nt = plan.nt;
    p.splits = plan.splits;
    p.stages = plan.stages;
    p.tiles_t = (p.T + p.nt - 1) / p.nt;
    p.status = static_cast<int32_t*>(ws);
    p.timeout_ns = L.timeout_ns;
    p.stall = L.flags & MOE_FFN_TEST_STALL0;
    const size_t smem = (size_t)p.stages * fx_stage_bytes(MODE == FF_SWIGLU, p.nt) + 1024;
    cudaError_t e = fx_prepare<MODE, A_MN>();
    if (e != cudaSuccess) return cuda_fail(e, what);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.M + 127) / 128 * p.tiles_t * p.splits));
    cfg.blockDim = dim3(GEMM_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)p.splits, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = p.splits > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, flex_kernel<MODE, A_MN>, p);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, what);
}
// Weights [M, K] (K-major, or stored [K, M]) and tokens [T, K] of operand pair i.
int fx_operands(FxArgs& p, int i, const void* w, int a_mn, const void* x, size_t M, size_t T, size_t K, int nt) {
    const int rc = ff_operand(&p.a[i], w, M, K, a_mn);
    return rc ? rc : ff_map(&p.b[i], x, T, K, (uint32_t)nt);
}
FxArgs fx_args(size_t M, size_t T, int kb0, int kb, void* out, int early) {
    FxArgs p;
    p.M = (int)M;
    p.T = (int)T;
    p.kb0 = kb0;
    p.kb = kb;
    p.out0 = static_cast<__nv_bfloat16*>(out);
    p.out1 = nullptr;
    p.gu = nullptr;
    p.early = early;
    return p;
}

// A dense launch over the tiles of products of two lengths, `cuttable` ones and `fixed` ones: in how many
// parts each cuttable tile goes, and how the units go round (ff_unit), the longer kind first.
struct FfSchedule {
    int parts, cut_last, extra;
    float us;
};
FfSchedule ff_schedule(int cuttable, int cuttable_kb, int fixed, int fixed_kb, int clusters) {
    auto tile = [](float work) {
        const float epi = US_DENSE_EPI[FK_PLAIN];
        return (work > epi ? work : epi) + US_DENSE_WAVE;
    };
    const float fixed_us = tile(fixed_kb * US_DENSE_KB);
    FfSchedule best{1, 0, 0, 1e30f};
    for (int parts = 1; parts <= 8; ++parts) {
        if (parts > 1 && (cuttable > FF_MAX_CUT / 2 || cuttable * parts > FF_MAX_CUT || parts * 4 > cuttable_kb)) break;
        const float part = (cuttable_kb + parts - 1) / parts * US_DENSE_KB;
        const float cut_us = parts > 1 ? part + US_CUT_ROUND : tile(part);
        const int cut_last = cut_us < fixed_us;
        const int n1 = cut_last ? fixed : cuttable * parts, n2 = cut_last ? cuttable * parts : fixed;
        const float t1 = cut_last ? fixed_us : cut_us, t2 = cut_last ? cut_us : fixed_us;
        const int rounds = n1 / clusters, high = n1 % clusters, low = clusters - high;
        const int most = high ? (int)(t1 / t2) + 1 : 0;
        for (int extra = 0; extra <= most && extra * low <= n2; ++extra) {
            const int left = n2 - extra * low, more = left / clusters, rest = left % clusters;
            const float end_low = rounds * t1 + (extra + more + (rest > 0)) * t2;
            const float end_high = high ? (rounds + 1) * t1 + (more + (rest > low)) * t2 : 0.0f;
            const float us = US_DENSE + (end_low > end_high ? end_low : end_high) + US_DENSE_EPI[FK_PLAIN] +
                             US_CUT_PART * (parts - 1);
            if (us < best.us) best = FfSchedule{parts, cut_last, extra, us};
        }
    }
    return best;
}

// The plans of a config's products. h for a backward pass (kept) and the hidden gradients (act) take the
// same kernel, because it fixes the layout in which g and u are kept.
struct FfPlans {
    int T, d, F, sms;
    FxPlan h, kept, act, down, dx;
    FfSchedule grad;  // of dx and the weight gradients in one launch, unless dx has a plan on flex_kernel
};
const FfPlans& ff_plans(const FfLayout& L, int sms) {
    static thread_local FfPlans last[4] = {};  // a program alternates between few configs
    static thread_local int turn = 0;
    const int T = (int)L.T, d = (int)L.d, F = (int)L.F;
    for (const FfPlans& p : last)
        if (p.T == T && p.d == d && p.F == F && p.sms == sms) return p;
    FfPlans& p = last[turn++ & 3];
    const int kd = (d + BK - 1) / BK, kf = (F + BK - 1) / BK;
    FxPlan kept = ff_choose_flex(F, T, kd, FK_H_KEPT, sms), act = ff_choose_flex(F, T, kd, FK_ACT, sms);
    const FxPlan dk = ff_dense(F, T, kd, FK_H_KEPT, sms), da = ff_dense(F, T, kd, FK_ACT, sms);
    if (dk.us + da.us < kept.us + act.us) {
        kept = dk;
        act = da;
    }
    p.T = T;
    p.d = d;
    p.F = F;
    p.sms = sms;
    p.h = ff_choose(F, T, kd, FK_H, sms);
    p.kept = kept;
    p.act = act;
    p.down = ff_choose(d, T, kf, FK_PLAIN, sms);
    // dx with the weight gradients in one launch, or on flex_kernel with them beside it
    p.dx = ff_choose_flex(d, T, 2 * kf, FK_PLAIN, sms);
    const int kt = (T + BK - 1) / BK;
    auto tiles = [](int m, int n) { return (m + FT_M - 1) / FT_M * ((n + FT_N - 1) / FT_N); };
    const int dw = 2 * tiles(F, d) + tiles(d, F);
    p.grad = ff_schedule(tiles(T, d), 2 * kf, dw, kt, sms / 2);
    if (p.grad.us <= p.dx.us + ff_cut(dw, kt, sms / 2).us + US_APART) p.dx.nt = 0;
    return p;
}

// A call's tensors: the address range of each, by name.
struct FfRange {
    const char* name;
    const void* ptr;
    size_t bytes;
};
// Refuses an output that shares memory with an input, or with an output after it in the list.
template <int NO, int NI>
int ff_apart(const FfRange (&outs)[NO], const FfRange (&ins)[NI]) {
    auto meet = [](const FfRange& a, const FfRange& b) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(a.ptr), q = reinterpret_cast<uintptr_t>(b.ptr);
        return p < q + b.bytes && q < p + a.bytes;
    };
    for (int i = 0; i < NO; ++i) {
        for (const FfRange& r : ins)
            if (meet(outs[i], r)) return fail(MOE_ERR_ARG, "%s overlaps %s", outs[i].name, r.name);
        for (int k = i + 1; k < NO; ++k)
            if (meet(outs[i], outs[k])) return fail(MOE_ERR_ARG, "%s overlaps %s", outs[i].name, outs[k].name);
    }
    return MOE_OK;
}

int ff_begin(const moe_ffn_config* c, void* ws, size_t ws_bytes, FfLayout* L, int* sms) {
    clear_error();
    int rc = ff_layout(c, L);
    if (rc) return rc;
    if (!ws) return fail(MOE_ERR_ARG, "workspace is NULL");
    if (!aligned(ws, 256)) return fail(MOE_ERR_ARG, "workspace must be 256-byte aligned");
    if (ws_bytes < L->ws_bytes) return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, L->ws_bytes);
    DeviceInfo di;
    if ((rc = device_info(&di))) return rc;
    *sms = di.sms;
    return di.supported ? MOE_OK : fail(MOE_ERR_DEVICE, "current device is not sm_103 (GB300)");
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

MOE_API int moe_ffn_workspace_size(const moe_ffn_config* c, size_t* bytes) {
    clear_error();
    FfLayout L;
    const int rc = ff_layout(c, &L);
    if (rc) return rc;
    if (!bytes) return fail(MOE_ERR_ARG, "bytes is NULL");
    *bytes = L.ws_bytes;
    return MOE_OK;
}

MOE_API int moe_ffn_saved_size(const moe_ffn_config* c, size_t* bytes) {
    clear_error();
    FfLayout L;
    const int rc = ff_layout(c, &L);
    if (rc) return rc;
    if (!bytes) return fail(MOE_ERR_ARG, "bytes is NULL");
    *bytes = L.saved_bytes;
    return MOE_OK;
}

MOE_API int moe_ffn_forward(const moe_ffn_config* c, const uint16_t* x, const uint16_t* W1, const uint16_t* W3,
                            const uint16_t* W2, uint16_t* y, void* saved, void* ws, size_t ws_bytes, void* stream) {
    FfLayout L;
    int sms = 0, rc = ff_begin(c, ws, ws_bytes, &L, &sms);
    if (rc) return rc;
    if (L.T == 0) return MOE_OK;
    if (!x || !W1 || !W3 || !W2 || !y) return fail(MOE_ERR_ARG, "NULL input or output pointer");
    if (!aligned(x, 16) || !aligned(W1, 16) || !aligned(W3, 16) || !aligned(W2, 16) || !aligned(y, 16))
        return fail(MOE_ERR_ARG, "x, W1, W3, W2, y must be 16-byte aligned");
    if (!aligned(saved, 256)) return fail(MOE_ERR_ARG, "saved must be 256-byte aligned");
    const size_t tokens = L.T * L.d * 2, matrix = L.F * L.d * 2;
    const FfRange outs[] = {{"y", y, tokens}}, ins[] = {{"W2", W2, matrix}, {"saved", saved, saved ? L.saved_bytes : 0}};
    if ((rc = ff_apart(outs, ins))) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t* s = static_cast<uint8_t*>(saved);
    uint8_t* h = s ? s + L.saved_h : static_cast<uint8_t*>(ws) + L.h;
    const int kd = (int)((L.d + BK - 1) / BK), kf = (int)((L.F + BK - 1) / BK);
    float* gu = s ? reinterpret_cast<float*>(s + L.saved_gu) : nullptr;
    const FfPlans& plans = ff_plans(L, sms);
    const FxPlan& up_plan = gu ? plans.kept : plans.h;
    if (up_plan.nt) {
        FxArgs p = fx_args(L.F, L.T, kd, kd, h, 0);
        p.gu = reinterpret_cast<float2*>(gu);
        if ((rc = fx_operands(p, 0, W1, 0, x, L.F, L.T, L.d, up_plan.nt))) return rc;
        if ((rc = fx_operands(p, 1, W3, 0, x, L.F, L.T, L.d, up_plan.nt))) return rc;
        if ((rc = fx_run<FF_SWIGLU, false>(p, up_plan, L, ws, st, "gate and up projections"))) return rc;
    } else {
        FfList up;
        FfProblem& p = up.add(x, 0, W1, 0, h, L.T, L.F, L.d);
        up.try_(ff_operand(&p.b[1], W3, L.F, L.d, 0));
        p.tiles_n = (int)((L.F + 127) / 128);  // 128 columns of g beside 128 of u
        p.whole = p.tiles_m * p.tiles_n;
        up.l.gu = gu;
        up.l.gu_cols = L.gu_cols;
        if ((rc = ff_run<FF_SWIGLU>(up, L, ws, st, "gate and up projections"))) return rc;
    }
    const FxPlan& down_plan = plans.down;
    if (down_plan.nt) {
        FxArgs p = fx_args(L.d, L.T, kf, kf, y, 1);
        if ((rc = fx_operands(p, 0, W2, 0, h, L.d, L.T, L.F, down_plan.nt))) return rc;
        return fx_run<FF_PLAIN, false>(p, down_plan, L, ws, st, "down projection");
    }
    FfList down;
    down.add(h, 0, W2, 0, y, L.T, L.d, L.F);
    return ff_run<FF_PLAIN>(down, L, ws, st, "down projection");
}

MOE_API int moe_ffn_backward(const moe_ffn_config* c, const uint16_t* x, const uint16_t* W1, const uint16_t* W3,
                             const uint16_t* W2, const uint16_t* dy, const void* saved, uint16_t* dx, uint16_t* dW1,
                             uint16_t* dW3, uint16_t* dW2, void* ws, size_t ws_bytes, void* stream) {
    FfLayout L;
    int sms = 0, rc = ff_begin(c, ws, ws_bytes, &L, &sms);
    if (rc) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!dW1 || !dW3 || !dW2) return fail(MOE_ERR_ARG, "NULL weight gradient pointer");
    if (!aligned(dW1, 16) || !aligned(dW3, 16) || !aligned(dW2, 16))
        return fail(MOE_ERR_ARG, "dW1, dW3, dW2 must be 16-byte aligned");
    if (L.T == 0) {
        cudaError_t e = cudaMemsetAsync(dW1, 0, L.F * L.d * 2, st);
        if (e == cudaSuccess) e = cudaMemsetAsync(dW3, 0, L.F * L.d * 2, st);
        if (e == cudaSuccess) e = cudaMemsetAsync(dW2, 0, L.F * L.d * 2, st);
        return e == cudaSuccess ? MOE_OK : cuda_fail(e, "clearing the weight gradients");
    }
    if (!x || !W1 || !W3 || !W2 || !dy || !saved || !dx) return fail(MOE_ERR_ARG, "NULL input or output pointer");
    if (!aligned(x, 16) || !aligned(W1, 16) || !aligned(W3, 16) || !aligned(W2, 16) || !aligned(dy, 16) ||
        !aligned(dx, 16))
        return fail(MOE_ERR_ARG, "x, W1, W3, W2, dy, dx must be 16-byte aligned");
    if (!aligned(saved, 256)) return fail(MOE_ERR_ARG, "saved must be 256-byte aligned");
    // dx is written beside the weight gradients, which read dy, x and saved, and beside the reads of W1 and W3
    const size_t tokens = L.T * L.d * 2, matrix = L.F * L.d * 2;
    const FfRange outs[] = {{"dx", dx, tokens}, {"dW1", dW1, matrix}, {"dW3", dW3, matrix}, {"dW2", dW2, matrix}};
    const FfRange ins[] = {{"x", x, tokens},   {"W1", W1, matrix},  {"W3", W3, matrix},
                           {"W2", W2, matrix}, {"dy", dy, tokens}, {"saved", saved, L.saved_bytes}};
    if ((rc = ff_apart(outs, ins))) return rc;
    const uint8_t* s = static_cast<const uint8_t*>(saved);
    const uint8_t* h = s + L.saved_h;
    uint8_t* dg = static_cast<uint8_t*>(ws) + L.dg;
    uint8_t* du = static_cast<uint8_t*>(ws) + L.du;
    const int kd = (int)((L.d + BK - 1) / BK), kf = (int)((L.F + BK - 1) / BK);
    float* gu = reinterpret_cast<float*>(const_cast<uint8_t*>(s) + L.saved_gu);
    const FfPlans& plans = ff_plans(L, sms);
    if (plans.act.nt) {
        const FxPlan& plan = plans.act;
        FxArgs p = fx_args(L.F, L.T, kd, kd, dg, 0);
        p.out1 = reinterpret_cast<__nv_bfloat16*>(du);
        p.gu = reinterpret_cast<float2*>(gu);
        if ((rc = fx_operands(p, 0, W2, 1, dy, L.F, L.T, L.d, plan.nt))) return rc;
        if ((rc = fx_run<FF_DACT, true>(p, plan, L, ws, st, "hidden gradients"))) return rc;
    } else {
        FfList act;
        FfProblem& p = act.add(dy, 0, W2, 1, dg, L.T, L.F, L.d);
        p.out[1] = reinterpret_cast<__nv_bfloat16*>(du);
        act.l.gu = gu;
        act.l.gu_cols = L.gu_cols;
        if ((rc = ff_run<FF_DACT>(act, L, ws, st, "hidden gradients"))) return rc;
    }
    FfList grad;
    const FxPlan& dx_plan = plans.dx;
    if (dx_plan.nt) {
        FxArgs p = fx_args(L.d, L.T, kf, 2 * kf, dx, 1);
        if ((rc = fx_operands(p, 0, W1, 1, dg, L.d, L.T, L.F, dx_plan.nt))) return rc;
        if ((rc = fx_operands(p, 1, W3, 1, du, L.d, L.T, L.F, dx_plan.nt))) return rc;
        if ((rc = fx_run<FF_PLAIN, true>(p, dx_plan, L, ws, st, "input gradients"))) return rc;
        grad.l.beside = 1;  // the weight gradients do not need dx
    }
    const FfSchedule& order = plans.grad;
    auto units = [&] {
        int n = 0;
        for (int i = 0; i < grad.l.count; ++i) n += grad.l.p[i].units();
        return n;
    };
    auto add_dx = [&] {
        FfProblem& p = grad.add(dg, 0, W1, 1, dx, L.T, L.d, L.F, du, W3);
        if (order.parts > 1) p.whole = 0;
        p.parts = order.parts;
    };
    if (!dx_plan.nt && !order.cut_last) add_dx();
    int first = units();
    grad.add(dg, 1, x, 1, dW1, L.F, L.d, L.T);
    grad.add(du, 1, x, 1, dW3, L.F, L.d, L.T);
    grad.add(dy, 1, h, 1, dW2, L.d, L.F, L.T);
    if (!dx_plan.nt && order.cut_last) {
        first = units();
        add_dx();
    }
    grad.l.first = first;  // none where dx has a launch of its own
    grad.l.extra = first ? order.extra : 0;
    return ff_run<FF_PLAIN>(grad, L, ws, st, "input and weight gradients");
}

MOE_API int moe_ffn_status(const moe_ffn_config* c, const void* ws, void* stream, int32_t* detail) {
    clear_error();
    FfLayout L;
    const int rc = ff_layout(c, &L);
    if (rc) return rc;
    if (!ws) return fail(MOE_ERR_ARG, "workspace is NULL");
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "stream synchronize");
    int32_t w[2] = {0, 0};
    e = cudaMemcpy(w, ws, sizeof(w), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_fail(e, "status read");
    if (detail) *detail = w[1];
    if (w[0] == ST_OK) return MOE_OK;
    return fail(MOE_ERR_TIMEOUT, "a bounded wait of the feed-forward block ran out (status %d, detail %d)", w[0], w[1]);
}

}  // extern "C"
