// Stage 5 over the 8-bit KV cache, tensor-core path (sm_103a): tree-masked
// GQA attention for more than 16 query rows per KV head.
//
// For sequence b and KV head hk the G = Hq/Hkv query heads of every tree slot
// form G*T query rows, in row blocks of 128. An item is a pair of row blocks
// with all keys; a worker (one CTA per SM) walks its pieces of items
// (kvq_sched.cuh) in key tiles of 64. Per tile t and row block g of the pair:
//   S = q K^T        tcgen05.mma kind::f8f6f4 straight from the codes: a row
//                    of q, scaled by a power of two to at most 256, is split
//                    into two e4m3 operands q = hi + lo (eight significant
//                    bits in all, those of bf16; elements below 2^-9 of the
//                    row's largest lose some), two MMAs at twice the fp16
//                    rate, by a small kernel before this one. (K to bf16 and q
//                    as it is: 945 against 703 us at 70B 32K then, for the
//                    conversion of K and the larger tiles in shared memory.)
//   P = softmax part four warps, one thread per row (TMEM lane = row, 64 key
//                    columns): K's block scale and q's row scale, tree mask,
//                    exponentials in the log2 domain against a reference
//                    maximum with V's block scale over a reference scale in
//                    the exponent, as fp16 pairs into tensor memory over S
//   O += P V         tcgen05.mma kind::f16, A = P from tensor memory, B = V as
//                    fp16 in shared memory (MN-major), converted from the
//                    tile's codes (exact, one conversion per two elements) by
//                    two warps of their own, once for both row blocks. P in
//                    e4m3 would spare that, at 2^-4 per weight instead of 2^-11.
// The reference maximum (scale) is raised, and O and the row sum rescaled in
// place, only when a tile's exceeds it by more than 2^8 (2^4), so the weights
// stay below 2^12. S is double buffered per row block: while one block's
// softmax works, the tensor pipe serves the other and the next tile. q of the
// next item arrives while the current one runs (double buffered). Codes
// arrive by TMA (128-byte swizzle) in rings of their own; mbarriers order
// everything and every wait is bounded.
//
// Bound by the tensor pipe: per tile and row block eight QK^T MMAs of 48
// cycles (N = 64 is bound by reading the operands from shared memory) and four
// PV MMAs of 64, so 1280 cycles for both blocks of a tile of some 1500 measured
// (8 sequences of 32K, 70B heads: 557 us in a captured graph, 560 to 580 call
// after call, by the card; 64 sequences of 8B: 121 us; one of 2048: 25 us). That
// holds while the two blocks' softmaxes run half a tile apart, as they do in this
// build: nothing here orders them. Builds of the same loop in which they ran
// together took 1900 (710 us; 743 us and 149 us at 8B with nothing changed but
// the kind of load of the sequences' lengths, so time this kernel after any
// change), and letting PV of one block wait for the other's QK^T did not part
// them (807 us). What was tried against the bound: QK^T over 128 keys at
// once (N = 128, two thirds of the cycles) leaves no second buffer of S, and
// waits for PV (857 us); S freed as soon as it is read, with P beside it, puts
// the copy's, QK^T's and softmax's latencies in one chain (678 us); half a row
// per softmax thread (24 warps of 80 registers, 730 against 701 us then);
// exponentials as polynomials on the FMA pipe (753 us); the weights against
// the last tile's maximum while this tile's is found (733 against 690 us).

#include "kvq_sched.cuh"

#include <cmath>

namespace eagle {
namespace {

constexpr int kBM = 128;
constexpr int kBN = 64;                  // keys per tile
constexpr int kSub = kBN / 16;           // 16-key groups of a tile: each lies in one scale block
constexpr int kHD = kKvqHeadDim;
constexpr int kTileQ = kBM * kHD;        // 16 KB: one e4m3 part of a row block's q
constexpr int kTile8 = kBN * kHD;        // 8 KB: a K or V tile of codes
constexpr int kTileV = kBN * kHD * 2;    // 16 KB: V as fp16, two halves of 64 columns
constexpr int kHalfV = kTileV / 2;
constexpr int kKStages = 4, kVStages = 3;  // tiles of codes in flight
constexpr int kScaleSlots = 8;
// Sixteen warps: 0 copies; 1, 2 QK^T of block 0, 1; 3, 4 PV of block 0, 1; 5, 6 converters; 7 scales;
// 8..11 and 12..15 softmax of block 0 and 1. (The scales as the copying warp's work made it the
// slowest of all: 1750 cycles a tile.)
constexpr int kWarpMma = 1, kWarpConv = 5, kWarpScale = 7, kWarpSoftmax = 8;
constexpr int kConvWarps = 2, kSoftmaxWarps = 8;
constexpr int kThreads = 32 * (kWarpSoftmax + kSoftmaxWarps);
constexpr int kSmemQ = 0;  // [item parity][row block][hi, lo]
constexpr int kSmemK = 8 * kTileQ;
constexpr int kSmemV8 = kSmemK + kKStages * kTile8;
constexpr int kSmemV = kSmemV8 + kVStages * kTile8;  // [tile parity]
constexpr int kSmem = kSmemV + 2 * kTileV + 1024;   // and alignment slack
constexpr int kTmemCols = 512;  // S of row block g, buffer b at 64 (2g + b) (P over it), O of block g at 256 + 128 g

// kind::f8f6f4, both operands e4m3 (type 0), fp32 accumulate; kind::f16 with both fp16 (type 0).
__host__ __device__ constexpr uint32_t idesc_type0(int M, int N, int b_mn_major) {
    return (1u << 4) | (static_cast<uint32_t>(b_mn_major) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}
// An MMA warp runs as one: every lane computes the same descriptors (in
// uniform registers) and one elected lane issues, by a predicate inside the
// instruction. Issued from a branch that one lane takes, each MMA moves its six
// operands into uniform registers first: about 110 cycles per instruction, three
// times what it computes (70B 32K: 1329 us).
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(e));
    return e;
}
__device__ __forceinline__ void mma_f8(uint32_t lead, uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, int accum) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(tmem_d),
        "l"(a), "l"(b), "r"(idesc), "r"(accum), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t lead, uint32_t tmem_d, uint32_t tmem_a, uint64_t b, uint32_t idesc,
                                           int accum) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(tmem_d),
        "r"(tmem_a), "l"(b), "r"(idesc), "r"(accum), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t lead, uint64_t* bar) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_u32(bar)),
        "r"(lead)
        : "memory");
}
// One lane's copy, issued like an MMA by the whole warp.
__device__ __forceinline__ void expect_tx(uint32_t lead, uint64_t* bar, uint32_t bytes) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n"
        " @q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}" ::"r"(smem_u32(bar)),
        "r"(bytes), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void copy_4d(uint32_t lead, uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                        uint64_t* bar) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %7, 0;\n"
        " @q cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];\n}" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar)), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void arrive(uint32_t lead, uint64_t* bar) {
    asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n @q mbarrier.arrive.shared::cta.b64 _, [%0];\n}" ::"r"(smem_u32(bar)),
                 "r"(lead)
                 : "memory");
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ float max16(const uint32_t* v) {
    auto f = [&](int i) { return __uint_as_float(v[i]); };
    const float a = fmax3(f(0), f(1), f(2)), b = fmax3(f(3), f(4), f(5)), c = fmax3(f(6), f(7), f(8));
    const float d = fmax3(f(9), f(10), f(11)), e = fmax3(f(12), f(13), f(14));
    return fmaxf(fmax3(a, b, c), fmax3(d, e, f(15)));
}

// Bounded waits of a whole warp. Every lane polls: tensor-memory instructions
// want the warp converged, which one lane's polls and a warp barrier do not
// promise. SLEEP: a short nap between polls, for the waits that are long
// anyway, so that idle warps leave issue slots and the barrier unit to the
// others. After a first timeout later waits are short, so that a failed launch
// still ends promptly (its results are meaningless then and the status says
// so; every role keeps its own order of arrivals, so nobody waits without bound).
struct Waiter {
    bool ok = true;
    template <bool SLEEP = true>
    __device__ __forceinline__ void poll(uint64_t* bar, int phase) {
        const uint32_t limit = ok ? (1u << 21) : 64u;
        for (uint32_t i = 0; i < limit; ++i) {
            if (mbar_try_wait(bar, phase & 1)) return;
            if (SLEEP) __nanosleep(32);
        }
        ok = false;
    }
    __device__ __forceinline__ void operator()(uint64_t* bar, int phase) {
        poll(bar, phase);
        __syncwarp();
    }
    // Two barriers: both first polls in flight together (each answer takes over 100 cycles).
    template <bool SLEEP = true>
    __device__ __forceinline__ void both(uint64_t* a, int pa, uint64_t* b, int pb) {
        const bool ra = mbar_try_wait(a, pa & 1), rb = mbar_try_wait(b, pb & 1);
        if (!ra) poll<SLEEP>(a, pa);
        if (!rb) poll<SLEEP>(b, pb);
        __syncwarp();
    }
};

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {  // a in the low byte
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(b), "f"(a));
    return d;
}

// n / d by the reciprocal 2^63 / d, rounded up: exact for all 32-bit n and d.
// (Three divisions a row took half of the kernel's instructions.)
struct Divisor {
    uint64_t m;
    explicit Divisor(int d) : m((uint64_t{1} << 63) / static_cast<uint64_t>(d) + 1) {}
    __device__ __forceinline__ uint32_t of(uint32_t n) const {
        return static_cast<uint32_t>(__umul64hi(m, static_cast<uint64_t>(n) << 1));
    }
};

// q as two e4m3 parts: s x = hi + lo for a row x, s the power of two that
// brings its largest element into [128, 256); the softmax's factor log2(e) /
// (s sqrt(128)). From [B][T][Hq][128] to [B][Hkv][hi, lo][G*T][128] and
// [B][Hkv][G*T]. Sixteen lanes take a row, two rows each (both loads first).
// Moves 4 bytes per element; at 8B b64, 31 MB each way. (In the attention
// kernel, by its converters behind their tiles, it held up each item by
// 11,000 cycles: the fence behind a converted tile waits for the loads of q
// in flight.) The first CTAs find where the attention's workers start.
constexpr int kSplitThreads = 256, kSplitPer = 2, kSplitRows = kSplitPer * kSplitThreads / 16;
__global__ void __launch_bounds__(kSplitThreads)
    kvq_split_q_kernel(const __nv_bfloat16* q, uint2* __restrict__ dst, float* __restrict__ fac, KvqRows rows,
                       Divisor by_Hq, Divisor by_T, Divisor by_G, int Hkv, uint32_t n, float scale_log2, KvqSched sched,
                       KvqCursor* __restrict__ cursors) {
    pdl_wait_prior();
    pdl_launch_dependents();
    constexpr int kStarts = kSplitThreads / 32;
    const int starts = (sched.workers + kStarts - 1) / kStarts;
    if (static_cast<int>(blockIdx.x) < starts) {
        const int w = blockIdx.x * kStarts + (threadIdx.x >> 5);
        KvqCursor c;
        c.init(sched, w);
        if (w < sched.workers && (threadIdx.x & 31) == 0) cursors[w] = c;
        return;
    }
    const int l16 = threadIdx.x & 15;
    const uint32_t i0 = (blockIdx.x - starts) * kSplitRows + (threadIdx.x >> 4);
    uint4 u[kSplitPer];
#pragma unroll
    for (int e = 0; e < kSplitPer; ++e) {
        const uint32_t i = i0 + e * (kSplitThreads / 16);
        u[e] = i < n ? ld_prior(reinterpret_cast<const uint4*>(q) + static_cast<size_t>(i) * (kHD / 8) + l16) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int e = 0; e < kSplitPer; ++e) {
        uint32_t mx = __vmaxu2(__vmaxu2(u[e].x & 0x7fff7fffu, u[e].y & 0x7fff7fffu),
                               __vmaxu2(u[e].z & 0x7fff7fffu, u[e].w & 0x7fff7fffu));
#pragma unroll
        for (int m = 1; m < 16; m <<= 1) mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, m));
        mx = max(mx & 0xffffu, mx >> 16);
        const float s = pow2_to(__uint_as_float(mx << 16), 7);
        // a row with an infinity becomes NaN as a whole: as e4m3 an infinity would be 448
        const float sx = mx < 0x7f80u ? s : NAN;
        const uint32_t w[4] = {u[e].x, u[e].y, u[e].z, u[e].w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float x = __uint_as_float(w[c] << 16) * sx, y = __uint_as_float(w[c] & 0xffff0000u) * sx;
            hi[c] = e4m3x2(x, y);
            const uint32_t h = e4m3_to_f16x2(hi[c]);
            const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h));
            lo[c] = e4m3x2(x - b.x, y - b.y);
        }
        const uint32_t i = i0 + e * (kSplitThreads / 16);
        if (i >= n) continue;
        const uint32_t bt = by_Hq.of(i), b = by_T.of(bt);
        const uint32_t h = i - bt * rows.Hq, t = bt - b * rows.T, hk = by_G.of(h);
        const uint32_t RT = rows.G * rows.T, r = t * rows.G + (h - hk * rows.G);
        const size_t bk = static_cast<size_t>(b) * Hkv + hk;
        dst[(2 * bk * RT + r) * 16 + l16] = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
        dst[((2 * bk + 1) * RT + r) * 16 + l16] = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
        if (l16 == 0) fac[bk * RT + r] = scale_log2 / s;
    }
}

// What the softmax needs of a tile's scales, per 16-key group.
struct alignas(16) TileScales {
    float k[kSub];   // K's scale
    float lv[kSub];  // log2 of V's scale over the reference (at least 2^-24)
    float iv[kSub];  // the reverse of that ratio
    float alpha;     // O's factor when the reference was raised for this tile, else 1
    float sref;      // the reference scale
    float pad[2];
};

__global__ void __launch_bounds__(kThreads, 1)
    kvq_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, KvqAttnParams p) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t bar_q_full[2], bar_q_empty[2], bar_k_full[kKStages], bar_k_empty[kKStages], bar_v8_full[kVStages],
        bar_v8_empty[kVStages], bar_v_full[2], bar_v_empty[2], bar_sc[kScaleSlots], bar_go[kScaleSlots], bar_s_full[2][2],
        bar_p_full[2][2], bar_pv_done[2][2];
    __shared__ uint32_t tmem_holder;
    __shared__ TileScales ts[kScaleSlots];
    __shared__ KvqCursor softmax_cur[kSoftmaxWarps];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int worker = blockIdx.x;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar_q_full[s], 1);
            mbar_init(&bar_q_empty[s], 2);
            mbar_init(&bar_v_full[s], kConvWarps);
            mbar_init(&bar_v_empty[s], 2);
            for (int b = 0; b < 2; ++b) {
                mbar_init(&bar_pv_done[s][b], 1);
                mbar_init(&bar_s_full[s][b], 1);
                mbar_init(&bar_p_full[s][b], 4);
            }
        }
        for (int s = 0; s < kKStages; ++s) {
            mbar_init(&bar_k_full[s], 1);
            mbar_init(&bar_k_empty[s], 2);
        }
        for (int s = 0; s < kVStages; ++s) {
            mbar_init(&bar_v8_full[s], 1);
            mbar_init(&bar_v8_empty[s], kConvWarps);
        }
        for (int s = 0; s < kScaleSlots; ++s) {
            mbar_init(&bar_sc[s], 1);
            mbar_init(&bar_go[s], 1);
        }
        fence_mbar_init();
    }
    if (threadIdx.x == 32 * kWarpConv) {  // the maps are parameters: no need to wait for the kernels before
        prefetch_map(&tm_q);
        prefetch_map(&tm_k);
        prefetch_map(&tm_v);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_holder)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // Of what this kernel reads, only the split of q's results (q's parts and factors, the cursors) were written
    // since its launch: the split lets it start behind its own wait. The rest may be read by __ldg.
    pdl_wait_prior();
    pdl_launch_dependents();
    KvqCursor cur;
    {
        static_assert(sizeof(KvqCursor) % 16 == 0, "whole 16-byte pieces");
        const int4* src = reinterpret_cast<const int4*>(p.cursors + worker);
        int4* dst = reinterpret_cast<int4*>(&cur);
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(KvqCursor) / 16); ++i) dst[i] = __ldcg(src + i);
    }
    KvqPiece it;
    Waiter wait;
    const int rows = p.G * p.s.T, n_blocks = (rows + kBM - 1) / kBM;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_holder;

    if (warp == 0) {
        // -------------------------------------------------------- copies ---
        // Step t: once the stages of tile t are free (both blocks' QK^T of tile t - 4
        // done, V of tile t - 3 converted), say that the slot of the scales of tile
        // t - 1 is free, and copy K and V of tile t. (The slot held tile t - 9's: V(t - 4)
        // was converted after both blocks' PV of tile t - 6.) The next item's q is
        // asked for once this item's fifth tile starts: the last item's QK^T are done by then.
        const uint32_t lead = elect_one(), base = smem_u32(smem);
        int t = 0, qi = 0, sk = 0, pk = 0, sv = 0, pv = 0;  // stages of tile t and their phases
        auto copy_q = [&](const KvqPiece& a, int i) {  // q of the i-th item
            if (i >= 2) wait(&bar_q_empty[i & 1], (i >> 1) - 1);
            if (__all_sync(0xffffffffu, wait.ok)) {
                const int hk = uniform(a.sub / p.n_items), block = uniform((a.sub - hk * p.n_items) * 2);
                const int n = min(2, n_blocks - block), w = uniform(a.b) * p.Hkv + hk;
                expect_tx(lead, &bar_q_full[i & 1], n * 2 * kTileQ);
                for (int h = 0; h < 2 * n; ++h)  // (row block, part); rows past the last are zeros
                    copy_4d(lead, base + kSmemQ + ((i & 1) * 4 + h) * kTileQ, &tm_q, 0, (block + (h >> 1)) * kBM, h & 1, w,
                            &bar_q_full[i & 1]);
            }
        };
        KvqPiece ahead;
        bool more = cur.next<true>(p.s, ahead);
        if (more) copy_q(ahead, 0);
        for (; uniform(more); ++qi) {
            it = ahead;
            more = cur.next<true>(p.s, ahead);
            const int hk = uniform(it.sub / p.n_items), b = uniform(it.b), j1 = uniform(it.t1), j0 = uniform(it.t0);
            for (int j = j0; j < j1; ++j, ++t) {
                if (t >= kKStages) wait.both(&bar_k_empty[sk], pk ^ 1, &bar_v8_empty[sv], pv ^ 1);
                else if (t >= kVStages) wait(&bar_v8_empty[sv], pv ^ 1);
                if (t > 0 && lane == 0) mbar_arrive(&bar_go[(t - 1) & (kScaleSlots - 1)]);
                __syncwarp();
                if (__all_sync(0xffffffffu, wait.ok)) {
                    expect_tx(lead, &bar_k_full[sk], kTile8);
                    copy_4d(lead, base + kSmemK + sk * kTile8, &tm_k, 0, hk, j * kBN, b, &bar_k_full[sk]);
                    expect_tx(lead, &bar_v8_full[sv], kTile8);
                    copy_4d(lead, base + kSmemV8 + sv * kTile8, &tm_v, 0, hk, j * kBN, b, &bar_v8_full[sv]);
                }
                if (++sk == kKStages) {
                    sk = 0;
                    pk ^= 1;
                }
                if (++sv == kVStages) {
                    sv = 0;
                    pv ^= 1;
                }
                if (more && j == min(j0 + 4, j1 - 1)) copy_q(ahead, qi + 1);
            }
        }
        if (t > 0 && lane == 0) mbar_arrive(&bar_go[(t - 1) & (kScaleSlots - 1)]);
        __syncwarp();
        if (!wait.ok) {  // the copies in flight land before the CTA's shared memory goes away
            if (lane == 0) raise_status(p.status, kDevTimeout);
            for (int s = 0; s < 2; ++s)
                for (int ph = 0; ph < 2; ++ph) mbar_wait(&bar_q_full[s], ph, 1u << 16);
            for (int s = 0; s < kVStages; ++s)
                for (int ph = 0; ph < 2; ++ph) mbar_wait(&bar_v8_full[s], ph, 1u << 16);
            for (int s = 0; s < kKStages; ++s)
                for (int ph = 0; ph < 2; ++ph) mbar_wait(&bar_k_full[s], ph, 1u << 16);
        }
        __syncwarp();
    } else if (warp < kWarpConv) {
        // --------------------------------------------------- MMA issuers ---
        // Per row block g one warp issues QK^T and one PV: a wait for a phase long
        // complete takes over 100 cycles, an MMA's issue about 20, and one warp
        // for both kinds took 2000 cycles a tile (for both blocks as well, 2660).
        // Tiles are numbered t over all of the worker's pieces, and u over those
        // in which the block has rows. QK(u) goes into S buffer u & 1, over the P
        // that PV(u - 2) reads, so it waits for that PV's completion. A piece's
        // first PV overwrites O: the softmax threads have read the previous piece's
        // O before they arrive for it. A PV's completion is told on one of two
        // barriers in turn: when the softmax waits for PV(u) the one before may
        // still be running, and a single barrier's parity would be taken for the
        // phase before.
        const uint32_t lead = elect_one();
        const uint32_t base = smem_u32(smem), tm = uniform(tmem);
        const int role = uniform(warp - kWarpMma);  // QK of block 0, 1, PV of block 0, 1
        const int g = role & 1;
        const uint32_t tS = tm + 128 * g, tO = tm + 256 + 128 * g;
        int t = 0, u = 0;
        int sk = 0, pk = 0;  // K stage of tile t and its phase
        auto next_k = [&]() {
            if (++sk == kKStages) {
                sk = 0;
                pk ^= 1;
            }
        };
        auto spin = [&](uint64_t* bar, int phase) {
            wait.poll<false>(bar, phase);
            __syncwarp();
        };
        if (role < 2) {
            constexpr uint32_t id_qk = idesc_type0(kBM, kBN, 0);
            for (int qi = 0;; ++qi) {
                const bool more = cur.next<true>(p.s, it);
                if (!uniform(more)) break;
                const int n_tiles = uniform(it.t1 - it.t0);
                const bool live = uniform((it.sub % p.n_items) * 2 + g) < n_blocks;
                const uint32_t aQ = base + kSmemQ + ((qi & 1) * 4 + 2 * g) * kTileQ;
                spin(&bar_q_full[qi & 1], qi >> 1);
                if (!live) {  // a block without rows: keep the shared barriers' counts, in step
                    for (int j = 0; j < n_tiles; ++j, ++t, next_k()) {
                        wait(&bar_k_full[sk], pk);
                        if (lane == 0) mbar_arrive(&bar_k_empty[sk]);
                    }
                    if (lane == 0) mbar_arrive(&bar_q_empty[qi & 1]);
                    continue;
                }
                for (int j = 0; j < n_tiles; ++j, ++t, ++u, next_k()) {
                    if (u >= 2) wait.both<false>(&bar_k_full[sk], pk, &bar_pv_done[g][u & 1], (u >> 1) - 1);
                    else spin(&bar_k_full[sk], pk);
                    tc_fence_after();
                    const uint32_t aK = base + kSmemK + sk * kTile8;
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)  // hi (0..3), lo (4..7); 32 elements of the head dimension each
                        mma_f8(lead, tS + 64 * (u & 1), smem_desc(aQ + (kk >> 2) * kTileQ + (kk & 3) * 32, 16, 1024),
                               smem_desc(aK + (kk & 3) * 32, 16, 1024), id_qk, kk > 0);
                    commit(lead, &bar_s_full[g][u & 1]);
                    commit(lead, &bar_k_empty[sk]);
                    if (j == n_tiles - 1) commit(lead, &bar_q_empty[qi & 1]);
                }
            }
            // the last commits' arrivals come before the CTA's shared memory goes away
            if (t > 0) wait(&bar_k_empty[(t - 1) % kKStages], (t - 1) / kKStages);
        } else {
            constexpr uint32_t id_pv = idesc_type0(kBM, kHD, 1);
            for (;;) {
                const bool more = cur.next<true>(p.s, it);
                if (!uniform(more)) break;
                const int n_tiles = uniform(it.t1 - it.t0);
                const bool live = uniform((it.sub % p.n_items) * 2 + g) < n_blocks;
                if (!live) {
                    for (int j = 0; j < n_tiles; ++j, ++t) {
                        wait(&bar_v_full[t & 1], t >> 1);
                        if (lane == 0) mbar_arrive(&bar_v_empty[t & 1]);
                    }
                    continue;
                }
                for (int j = 0; j < n_tiles; ++j, ++t, ++u) {
                    wait.both<false>(&bar_v_full[t & 1], t >> 1, &bar_p_full[g][u & 1], u >> 1);
                    tc_fence_after();
                    const uint32_t aV = base + kSmemV + (t & 1) * kTileV;
#pragma unroll
                    for (int kk = 0; kk < kBN / 16; ++kk)  // A = P from TMEM: 16 keys = 8 columns per MMA
                        mma_f16_ts(lead, tO, tS + 64 * (u & 1) + kk * 8, smem_desc(aV + kk * 2048, kHalfV, 1024), id_pv,
                                   (j > 0 || kk > 0) ? 1 : 0);
                    commit(lead, &bar_pv_done[g][u & 1]);
                    commit(lead, &bar_v_empty[t & 1]);
                }
            }
            if (t > 0) wait(&bar_v_empty[(t - 1) & 1], (t - 1) >> 1);
        }
        if (!wait.ok) raise_status(p.status, kDevTimeout);
    } else if (warp < kWarpScale) {
        // ----------------------------------------------------- converters ---
        const int cw = warp - kWarpConv;
        const uint32_t base = smem_u32(smem);
        int t = 0, st = 0, ph = 0;  // the stage of codes and its phase
        while (cur.next<true>(p.s, it))
            for (int j = it.t0; j < it.t1; ++j, ++t) {
                const int b = t & 1;
                if (t >= 2) wait.both(&bar_v_empty[b], (t >> 1) - 1, &bar_v8_full[st], ph);
                else wait(&bar_v8_full[st], ph);
                uint4 u[8];  // chunks cw, cw + 2, .. of 16 columns, two keys each
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int key = lane + 32 * (e & 1), c16 = cw + kConvWarps * (e >> 1);
                    u[e] = lds128(base + kSmemV8 + st * kTile8 + key * kHD + ((c16 ^ (key & 7)) << 4));
                    // keys that no row can see may hold anything (even NaN): 0 * V has to stay 0
                    if (j * kBN + key >= it.nkeys) u[e] = make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int key = lane + 32 * (e & 1), c16 = cw + kConvWarps * (e >> 1);
                    const uint32_t dst = base + kSmemV + b * kTileV + (c16 >> 2) * kHalfV + key * 128;
                    const int c = 2 * (c16 & 3);
                    sts128(dst + ((c ^ (key & 7)) << 4), make_uint4(e4m3_to_f16x2(u[e].x), e4m3_to_f16x2(u[e].x >> 16),
                                                                    e4m3_to_f16x2(u[e].y), e4m3_to_f16x2(u[e].y >> 16)));
                    sts128(dst + (((c + 1) ^ (key & 7)) << 4), make_uint4(e4m3_to_f16x2(u[e].z), e4m3_to_f16x2(u[e].z >> 16),
                                                                          e4m3_to_f16x2(u[e].w), e4m3_to_f16x2(u[e].w >> 16)));
                }
                fence_proxy_async_smem();  // the MMA reads V through the async proxy
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar_v8_empty[st]);
                    mbar_arrive(&bar_v_full[b]);
                }
                if (++st == kVStages) {
                    st = 0;
                    ph ^= 1;
                }
            }
        if (!wait.ok) raise_status(p.status, kDevTimeout);
    } else if (warp == kWarpScale) {
        // -------------------------------------------------------- scales ---
        // The softmax's scales of a tile, read a tile ahead (the fence behind a
        // converter's tile would wait for them; a QK warp was late for its next tile).
        // Lanes 0..3 hold K's scales of a tile's 16-key groups, 4..7 V's.
        int t = 0;
        float last_scale = 0.0f, sref = 0.0f, inv_sref = 0.0f;
        auto give = [&](int tile) {
            // V's reference scale: the piece's first tile's largest, raised by more than 2^4 only
            float vm = lane >= kSub && lane < 2 * kSub ? last_scale : 0.0f;
            vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, 1));
            vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, 2));
            vm = fmaxf(__shfl_sync(0xffffffffu, vm, kSub), kKvqMinRef);
            float alpha = 1.0f;
            if (vm > 16.0f * sref) {
                if (sref > 0.0f) alpha = sref / vm;
                sref = vm;
                inv_sref = 1.0f / vm;
            }
            const float ratio = fmaxf(last_scale * inv_sref, 0x1p-24f);
            const float lv = __log2f(ratio), iv = __frcp_rn(ratio);
            const int slot = tile & (kScaleSlots - 1);
            wait(&bar_go[slot], tile / kScaleSlots);
            TileScales& o = ts[slot];
            if (lane < 2 * kSub) (&o.k[0])[lane] = lane < kSub ? last_scale : lv;  // k, then lv
            if (lane >= kSub && lane < 2 * kSub) o.iv[lane - kSub] = iv;
            if (lane == 0) o.alpha = alpha;
            if (lane == 1) o.sref = sref;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_sc[slot]);
            __syncwarp();
        };
        int qi = 0;
        for (; cur.next<true>(p.s, it); ++qi) {
            const int hk = it.sub / p.n_items;
            const float* src = (lane < kSub ? p.k_scale : p.v_scale) + it.b * p.s_seq + hk;
            const int last = (it.nkeys - 1) >> p.blk_shift;
            for (int j = it.t0; j < it.t1; ++j, ++t) {
                float own = 0.0f;
                if (lane < 2 * kSub) own = __ldg(src + min((j * kBN + 16 * (lane & 3)) >> p.blk_shift, last) * p.s_blk);
                if (t > 0) give(t - 1);
                if (j == it.t0) sref = 0.0f;  // the tile just given was the last piece's
                last_scale = own;
            }
        }
        if (t > 0) give(t - 1);
        // The QK warps' commits on the last item's q, which nobody else waits for, arrive before the CTA's shared
        // memory goes away. (Its q was copied, so the barrier's phase before is over.)
        if (qi > 0) wait(&bar_q_empty[(qi - 1) & 1], (qi - 1) >> 1);
        if (!wait.ok && lane == 0) raise_status(p.status, kDevTimeout);
    } else {
        // ------------------------------------------------------ softmax ---
        // Four warps per row block; warp w serves TMEM lane quarter w % 4, one
        // thread per row.
        const int g = (warp - kWarpSoftmax) >> 2;
        const int q4 = warp & 3;
        const int r = (q4 << 5) | lane;   // row of the block = TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
        const uint32_t o_cols = tmem + 256 + 128 * g + lane_off;
        const uint32_t lead = elect_one();
        int t = 0, tg = 0;
        int4 cut = make_int4(0, 0, 0, 0);
        // The cursor waits in shared memory while a piece is worked on: a tile needs the registers.
        KvqCursor& own = softmax_cur[warp - kWarpSoftmax];
        if (lane == 0) own = cur;
        __syncwarp();
        auto next_piece = [&]() {
            KvqCursor c = own;
            __syncwarp();
            const bool more = c.next<true>(p.s, it);
            if (lane == 0) own = c;
            __syncwarp();
            return more;
        };
        kvq_zero_bad<true>(p.s, p.Hq, p.out, p.status, worker, threadIdx.x - kWarpSoftmax * 32, kSoftmaxWarps * 32);
        while (next_piece()) {
            if (it.np) cut = kvq_cut(it);
            const int hk = it.sub / p.n_items, block = (it.sub - hk * p.n_items) * 2 + g;
            const int nt = it.t1 - it.t0;
            if (block >= n_blocks) {  // the last pair of an odd number of row blocks: nothing to do for this one
                t += nt;
                continue;
            }
            int slot;
            const int64_t row = p.rows.row(it.b, hk, block * kBM + r, &slot);
            const bool row_live = row >= 0;
            // a quarter without rows of the problem does no arithmetic
            const bool quarter_live = __any_sync(0xffffffffu, row_live);
            const uint32_t* mrow =
                p.mask ? p.mask + (static_cast<size_t>(it.b) * p.s.T + (row_live ? slot : 0)) * p.W : nullptr;
            const int L = it.L, n = it.n;
            const float fac =
                row_live ? ld_prior(p.q_fac + (static_cast<size_t>(it.b) * p.Hkv + hk) * rows + block * kBM + r) : 0.0f;
            // word w of the row's mask
            auto word = [&](int w) {
                if (w >= p.W) return 0u;
                if (mrow) return __ldg(mrow + w);
                return slot >= 32 * w + 31 ? ~0u : slot < 32 * w ? 0u : (2u << (slot - 32 * w)) - 1u;
            };
            float m_use = 0.0f, l = 0.0f, sref = 0.0f;
            bool seen = false;
            // S of the piece's first tile before its scales are looked at: behind a piece without rows for
            // this block the scales' barrier may be phases back, and its parity be taken for this
            // tile's; S of a tile says that the tiles up to the sixth before it have theirs.
            wait(&bar_s_full[g][tg & 1], tg >> 1);
            for (int j = it.t0; j < it.t1; ++j, ++t, ++tg) {
                const int key0 = j * kBN;
                const uint32_t s_cols = tmem + 64 * (2 * g + (tg & 1)) + lane_off;
                wait.both(&bar_sc[t & (kScaleSlots - 1)], t / kScaleSlots, &bar_s_full[g][tg & 1], tg >> 1);
                tc_fence_after();
                if (quarter_live) {
                    const TileScales& sc = ts[t & (kScaleSlots - 1)];
                    const float4 k4 = *reinterpret_cast<const float4*>(sc.k), lv4 = *reinterpret_cast<const float4*>(sc.lv);
                    const float4 iv4 = *reinterpret_cast<const float4*>(sc.iv);
                    float k[kSub] = {k4.x * fac, k4.y * fac, k4.z * fac, k4.w * fac};
                    const float lv[kSub] = {lv4.x, lv4.y, lv4.z, lv4.w}, iv[kSub] = {iv4.x, iv4.y, iv4.z, iv4.w};
                    float alpha = sc.alpha;
                    sref = sc.sref;
                    uint32_t s[kBN];
                    tmem_ld64(s_cols, s);
                    // visibility of 32 keys at a time: prefix keys, then tree slots in the row's mask
                    if (key0 + kBN > L) {
                        uint32_t vis[2];
#pragma unroll
                        for (int hq = 0; hq < 2; ++hq) {
                            const int kb = key0 + 32 * hq;
                            const int npre = min(32, L - kb);  // keys of the 32 inside the prefix
                            const uint32_t pre = npre > 0 ? 0xffffffffu >> (32 - npre) : 0u;
                            const int j0 = kb - L;  // slot of the first key (may be negative)
                            const int lo = j0 < 0 ? 0 : j0;
                            const int w0 = lo >> 5, sh = lo & 31;
                            uint32_t win = word(w0) >> sh;
                            if (sh) win |= word(w0 + 1) << (32 - sh);
                            const int limit = n - lo;  // slots j >= n are never visible
                            if (limit <= 0) win = 0u;
                            else if (limit < 32) win &= (1u << limit) - 1u;
                            uint32_t tree = j0 < 0 ? (win << (-j0 & 31)) : win;
                            if (j0 <= -32) tree = 0u;
                            vis[hq] = pre | tree;
                        }
#pragma unroll
                        for (int e = 0; e < kBN; ++e) s[e] = ((vis[e >> 5] >> (e & 31)) & 1u) ? s[e] : 0xff800000u;
                        // -inf times a product that underflowed to 0 would be NaN (a row of zeros has the factor
                        // 2^-129, a block of zeros the scale 2^-126): above 0, a score changes by less than 2^-125
#pragma unroll
                        for (int e = 0; e < kSub; ++e) k[e] = fmaxf(k[e], 0x1p-149f);
                    }
                    const float mx = fmaxf(fmaxf(max16(s) * k[0], max16(s + 16) * k[1]),
                                           fmaxf(max16(s + 32) * k[2], max16(s + 48) * k[3]));  // the scales are positive
                    bool rescale = alpha != 1.0f;
                    if (mx > -INFINITY) {
                        if (!seen) {
                            m_use = mx;  // l is still zero (and so is the row of O)
                            seen = true;
                        } else if (mx > m_use + 8.0f) {
                            const float a = ex2_approx(m_use - mx);
                            m_use = mx;
                            l *= a;
                            alpha *= a;
                            rescale = true;
                        }
                    }
                    // (the vote here: its answer is not needed before P is written)
                    const bool any_rescale = __any_sync(0xffffffffu, rescale);
                    // P = 2^(s k - m_use + lv), two per packed multiply-add; the row sum takes the
                    // reverse of V's ratio. P as fp16 pairs over the first 32 columns of S.
                    // (A group's arguments, then its exponentials, then the last group's sums and
                    // pairs, in place: taken pair by pair every step waited for the one before.)
                    auto arguments = [&](int q) {
                        const float c = lv[q] - m_use;
                        const uint64_t k2 = f2_pack(k[q], k[q]), c2 = f2_pack(c, c);
#pragma unroll
                        for (int e = 16 * q; e < 16 * q + 16; e += 2) {
                            const uint64_t z = f2_fma((static_cast<uint64_t>(s[e + 1]) << 32) | s[e], k2, c2);
                            s[e] = __float_as_uint(f2_lo(z));
                            s[e + 1] = __float_as_uint(f2_hi(z));
                        }
                    };
                    auto exponentials = [&](int q) {
#pragma unroll
                        for (int e = 16 * q; e < 16 * q + 16; ++e) s[e] = __float_as_uint(ex2_approx(__uint_as_float(s[e])));
                    };
                    auto sum_and_pack = [&](int q) {
                        uint64_t a[2];
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const uint64_t w = (static_cast<uint64_t>(s[16 * q + e + 1]) << 32) | s[16 * q + e];
                            a[(e >> 1) & 1] = e < 4 ? w : f2_add(a[(e >> 1) & 1], w);
                        }
                        const uint64_t a2 = f2_add(a[0], a[1]);
                        l = fmaf(f2_lo(a2) + f2_hi(a2), iv[q], l);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            s[8 * q + e] = pack_f16(__uint_as_float(s[16 * q + 2 * e]), __uint_as_float(s[16 * q + 2 * e + 1]));
                    };
                    arguments(0);
#pragma unroll
                    for (int q = 0; q < kSub; ++q) {
                        if (q + 1 < kSub) arguments(q + 1);
                        exponentials(q);
                        if (q > 0) sum_and_pack(q - 1);
                    }
                    sum_and_pack(kSub - 1);
                    __syncwarp();  // the rows took different branches; tensor-memory accesses are the whole warp's
                    tmem_st32(s_cols, reinterpret_cast<const float*>(s));
                    // Rescaling O needs PV of the previous tile done (this tile's PV waits for
                    // this warp's arrival below). tcgen05.ld/st are warp-collective: rescale if
                    // any row of the warp needs it (alpha = 1 for the others).
                    if (j > it.t0 && any_rescale) {
                        wait(&bar_pv_done[g][(tg - 1) & 1], (tg - 1) >> 1);
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            float o[32];
                            tmem_ld32(o_cols + 32 * c, o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= alpha;
                            tmem_st32(o_cols + 32 * c, o);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                arrive(lead, &bar_p_full[g][tg & 1]);
            }
            // ----------------------------------------------------- epilogue ---
            wait(&bar_pv_done[g][(tg - 1) & 1], (tg - 1) >> 1);
            tc_fence_after();
            if (!quarter_live) continue;
            const bool any = row_live && seen && l > 0.0f && wait.ok;
            const bool whole = it.whole();
            const bool live = any && (!whole || slot < n);  // unused slots: zeros
            const float f = !live ? 0.0f : whole ? sref / l : sref;
            const size_t part_slot = it.slot(worker);
            const int prow = g * kBM + r;
            float4* part = reinterpret_cast<float4*>(p.part.o) + part_slot * (kHD / 4) * p.part.rows + prow;
            // whole: neighbouring lanes store 32 bytes of one row together (full sectors)
            const int64_t other = static_cast<int64_t>(shfl_xor_u64(static_cast<uint64_t>(row), 1));
            const bool odd = lane & 1;
            const int64_t row_e = odd ? other : row, row_o = odd ? row : other;  // the even lane's row, the odd one's
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                float o[32];
                __syncwarp();
                tmem_ld32(o_cols + 32 * c, o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = live ? o[e] * f : 0.0f;
                if (whole) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // 16 columns: chunks of 8 columns, this lane's x and y
                        uint4 x = make_uint4(pack_bf16(o[16 * h], o[16 * h + 1]), pack_bf16(o[16 * h + 2], o[16 * h + 3]),
                                             pack_bf16(o[16 * h + 4], o[16 * h + 5]), pack_bf16(o[16 * h + 6], o[16 * h + 7]));
                        uint4 y = make_uint4(pack_bf16(o[16 * h + 8], o[16 * h + 9]), pack_bf16(o[16 * h + 10], o[16 * h + 11]),
                                             pack_bf16(o[16 * h + 12], o[16 * h + 13]),
                                             pack_bf16(o[16 * h + 14], o[16 * h + 15]));
                        uint4 give = odd ? x : y, got;  // the even lane keeps x of its row and gets x of the odd one's
                        got.x = __shfl_xor_sync(0xffffffffu, give.x, 1);
                        got.y = __shfl_xor_sync(0xffffffffu, give.y, 1);
                        got.z = __shfl_xor_sync(0xffffffffu, give.z, 1);
                        got.w = __shfl_xor_sync(0xffffffffu, give.w, 1);
                        const int col = 32 * c + 16 * h + (odd ? 8 : 0);
                        if (row_e >= 0) *reinterpret_cast<uint4*>(p.out + row_e * kHD + col) = odd ? got : x;
                        if (row_o >= 0) *reinterpret_cast<uint4*>(p.out + row_o * kHD + col) = odd ? y : got;
                    }
                } else if (row_live) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        part[static_cast<size_t>(8 * c + q) * p.part.rows] =
                            make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                }
            }
            if (!whole && row_live)
                // (a sum that is NaN goes into the merge as it is: the whole row is zero then, not this piece left out)
                reinterpret_cast<float2*>(p.part.ml)[part_slot * p.part.rows + prow] =
                    make_float2(seen ? m_use : -INFINITY, wait.ok ? l : 0.0f);
            tc_fence_before();
        }
        if (!wait.ok) raise_status(p.status, kDevTimeout);
        if (threadIdx.x == kWarpSoftmax * 32) p.part.cut[worker] = cut;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// The cut item that worker w began (blockIdx.x), from its pieces i: worker w's
// in slot 2w + 1, w + i's in slot 2 (w + i). A warp takes eight rows; a lane
// one row and every fourth column group, so that the reads of the pieces are
// 128 bytes wide and the row's stores 32.
constexpr int kMergeWarps = 4;
__global__ void __launch_bounds__(kMergeWarps * 32) kvq_merge_rows_kernel(KvqMergeParams p) {
    const int lane = threadIdx.x & 31;
    const int r = (blockIdx.y * kMergeWarps + (threadIdx.x >> 5)) * 8 + (lane & 7), cg = lane >> 3;
    const int w = blockIdx.x;
    pdl_wait_prior();
    pdl_launch_dependents();
    const int4 c = __ldcg(p.part.cut + w);
    if (c.x == 0) return;
    const int hk = c.z / p.n_items;
    int slot;
    const int64_t row = p.rows.row(c.y, hk, (c.z - hk * p.n_items) * 2 * kBM + r, &slot);
    if (row < 0) return;
    const float2* ml = reinterpret_cast<const float2*>(p.part.ml);
    const float4* po = reinterpret_cast<const float4*>(p.part.o);
    RowSum<8> s;
#pragma unroll 2
    for (int i = 0; i < c.x; ++i) {
        const size_t at = i == 0 ? 2 * w + 1 : 2 * (w + i);
        const float2 a = __ldcg(ml + at * p.part.rows + r);
        float4 x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __ldcg(po + (at * (kHD / 4) + cg + 4 * e) * p.part.rows + r);
        s.add(a.x, a.y, x);
    }
    const bool live = slot < c.w && s.l > 0.0f;
    const float inv = live ? 1.0f / s.l : 0.0f;
    uint2* dst = reinterpret_cast<uint2*>(p.out + row * kHD);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        dst[cg + 4 * e] = live ? make_uint2(pack_bf16(s.o[e].x * inv, s.o[e].y * inv), pack_bf16(s.o[e].z * inv, s.o[e].w * inv))
                               : make_uint2(0u, 0u);
}

// ------------------------------------------------------------- host side ---

struct Plan {
    KvqSched s;
    int G, n_items, rows;
    bool decode;
    size_t off_cut, off_cur, off_ml, off_o, off_q, off_fac, bytes;
};

// Up to 16 query rows per KV head: the decode kernel, a worker per warp;
// more: the tensor-core kernel, a worker per CTA. A rule on rows because the
// first keeps 16 x 128 sums in a warp's registers.
Plan make_plan(const KvqDims& kv, int T) {
    Plan pl{};
    pl.G = kv.Hq / kv.Hkv;
    const int rows = pl.G * T;
    pl.decode = rows <= kKvqDecodeRows;
    if (pl.decode) {
        pl.n_items = 1;
        pl.rows = rows;
        pl.s = kvq_decode_sched(kv.B, T, kv.max_len, kv.Hkv, rows);
    } else {
        pl.n_items = (rows + 2 * kBM - 1) / (2 * kBM);
        pl.rows = 2 * kBM;
        // a tile with one block costs three quarters of one with two; a start and an end six tiles
        const int blocks = (rows + kBM - 1) / kBM;
        pl.s = KvqSched{nullptr, nullptr, kv.B, T, kv.max_len, kv.Hkv, pl.n_items, kBN, 24, 4, blocks % 2 ? 3 : 4, kKvqSms, 32};
    }
    const size_t slots = 2 * static_cast<size_t>(pl.s.workers) * pl.rows;
    pl.off_cut = 256;
    pl.off_cur = align_up(pl.off_cut + pl.s.workers * sizeof(int4), 256);
    pl.off_ml = align_up(pl.off_cur + (pl.decode ? 0 : pl.s.workers * sizeof(KvqCursor)), 256);
    pl.off_o = align_up(pl.off_ml + slots * 2 * sizeof(float), 256);
    pl.off_q = align_up(pl.off_o + slots * kHD * sizeof(float), 256);
    const size_t q_rows = pl.decode ? 0 : static_cast<size_t>(kv.B) * kv.Hkv * rows;
    pl.off_fac = pl.off_q + q_rows * 2 * kHD;
    pl.bytes = align_up(pl.off_fac + q_rows * sizeof(float), 256);
    return pl;
}

}  // namespace

size_t kvq_attention_ws_bytes(const KvqDims& kv, int T) { return make_plan(kv, T).bytes; }

cudaError_t launch_kvq_attention(const KvqDims& kv, int T, const void* q, const void* codes, const float* scales,
                                 int layer, const int32_t* prefix_len, const uint32_t* mask, const int32_t* n_tree,
                                 void* out, void* ws, cudaStream_t stream) {
    Plan pl = make_plan(kv, T);
    pl.s.prefix_len = prefix_len;
    pl.s.n_tree = n_tree;
    char* w = static_cast<char*>(ws);
    KvqAttnParams p{};
    p.s = pl.s;
    p.part = KvqPartials{reinterpret_cast<float*>(w + pl.off_o), reinterpret_cast<float*>(w + pl.off_ml),
                         reinterpret_cast<int4*>(w + pl.off_cut), pl.rows};
    p.rows = KvqRows{pl.G, T, kv.Hq};
    p.q_fac = reinterpret_cast<const float*>(w + pl.off_fac);
    p.cursors = reinterpret_cast<const KvqCursor*>(w + pl.off_cur);
    p.Hq = kv.Hq;
    p.Hkv = kv.Hkv;
    p.G = pl.G;
    p.n_items = pl.n_items;
    p.W = (T + 31) / 32;
    p.blk_shift = kv.block == 16 ? 4 : kv.block == 32 ? 5 : kv.block == 64 ? 6 : 7;
    p.s_seq = kv.s_seq;
    p.s_blk = kv.s_blk;
    p.k_scale = scales + layer * kv.s_layer;
    p.v_scale = p.k_scale + kv.s_kv;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.mask = mask;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.status = reinterpret_cast<int*>(w);
    p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(kHD)));
    const char* kbase = static_cast<const char*>(codes) + static_cast<int64_t>(layer) * kv.layer_stride;
    const char* vbase = kbase + kv.kv_stride;
    const KvqMergeParams mp{p.part, p.rows, pl.s.workers, p.n_items, p.out};
    if (pl.decode) {
        cudaError_t e = launch_kvq_decode(kv, p, kbase, vbase, stream);
        return e != cudaSuccess ? e : launch_kvq_merge_decode(mp, stream);
    }
    CUtensorMap tq, tk, tv;
    const int rows = pl.G * T;
    {  // (128 bytes, row, part, (sequence, KV head))
        auto fn = tensor_map_encode_fn();
        if (!fn) return cudaErrorInvalidValue;
        const cuuint64_t dims[4] = {kHD, static_cast<cuuint64_t>(rows), 2, static_cast<cuuint64_t>(kv.B) * kv.Hkv};
        const cuuint64_t strides[3] = {kHD, static_cast<cuuint64_t>(kHD) * rows, static_cast<cuuint64_t>(kHD) * rows * 2};
        const cuuint32_t box[4] = {kHD, kBM, 1, 1}, estride[4] = {1, 1, 1, 1};
        if (fn(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, w + pl.off_q, dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    if (!make_map_codes(&tk, kbase, kv, kBN) || !make_map_codes(&tv, vbase, kv, kBN)) return cudaErrorInvalidValue;
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kvq_attn_kernel), kSmem);
    if (e != cudaSuccess) return e;
    const int64_t q_rows = static_cast<int64_t>(kv.B) * T * kv.Hq;
    if (q_rows > INT32_MAX) return cudaErrorInvalidValue;  // half a terabyte of q
    e = launch_pdl(kvq_split_q_kernel, dim3(static_cast<unsigned>((q_rows + kSplitRows - 1) / kSplitRows + (pl.s.workers + kSplitThreads / 32 - 1) / (kSplitThreads / 32))), dim3(kSplitThreads), 0,
                   stream, p.q, reinterpret_cast<uint2*>(w + pl.off_q), reinterpret_cast<float*>(w + pl.off_fac), p.rows,
                   Divisor(kv.Hq), Divisor(T), Divisor(pl.G), kv.Hkv, static_cast<uint32_t>(q_rows), p.scale_log2, p.s, reinterpret_cast<KvqCursor*>(w + pl.off_cur));
    if (e != cudaSuccess) return e;
    e = launch_pdl(kvq_attn_kernel, dim3(pl.s.workers), dim3(kThreads), kSmem, stream, tq, tk, tv, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(kvq_merge_rows_kernel, dim3(pl.s.workers, pl.rows / (8 * kMergeWarps)), dim3(kMergeWarps * 32), 0, stream,
                      mp);
}

}  // namespace eagle
