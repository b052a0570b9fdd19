// Stage 5 over the 8-bit KV cache, tensor-core path (sm_103a): tree-masked
// GQA attention for more than 16 query rows per KV head.
//
// For sequence b and KV head hk the G = Hq/Hkv query heads of every tree slot
// form G*T query rows (row r <-> slot r / G, head hk*G + r % G), in row blocks
// of 128. A worker (one of two CTAs per SM) walks its pieces of (sequence,
// head, row block) items (kvq_sched.cuh) in key tiles of 64; per tile t:
//   S = q K^T        tcgen05.mma kind::f8f6f4 straight from the codes: a row
//                    of q, scaled by a power of two to at most 256, is split
//                    into two e4m3 operands q = hi + lo (eight significant
//                    bits in all, those of bf16; elements below 2^-9 of the
//                    row's largest lose some), two MMAs at twice the fp16
//                    rate. K needs no conversion and its tile is half the size.
//   P = softmax part eight warps, two threads per row (TMEM lane = row, 32 key
//                    columns each): K's block scale and q's row scale, tree
//                    mask, exponentials in the log2 domain against a reference
//                    maximum, times V's block scale over a reference scale,
//                    as fp16 pairs into tensor memory over the S buffer
//   O += P V         tcgen05.mma kind::f16, A = P from tensor memory, B = V as
//                    fp16 in shared memory (MN-major), which the softmax warps
//                    convert from the tile's codes (exact, one conversion per
//                    two elements) before they wait for S. P in e4m3 would
//                    spare that, at 2^-4 per weight instead of 2^-11.
// The reference maximum (scale) is raised, and O and the row sum rescaled in
// place, only when a tile's exceeds it by more than 2^8 (2^4), so the weights
// stay below 2^12. S is double buffered, QK^T of tile t+1 runs while the
// softmax works on tile t; the second CTA of the SM fills the tensor pipe
// meanwhile. Codes arrive by TMA (128-byte swizzle) in rings of their own;
// mbarriers order everything and every wait is bounded.

#include "kvq_sched.cuh"

#include <cmath>
#include <mutex>

namespace eagle {
namespace {

constexpr int kBM = 128;
constexpr int kBN = 64;                  // keys per tile
constexpr int kHD = kKvqHeadDim;
constexpr int kTileQ = kBM * kHD;        // 16 KB: one e4m3 part of q
constexpr int kTile8 = kBN * kHD;        // 8 KB: a K or V tile of codes
constexpr int kTileV = kBN * kHD * 2;    // 16 KB: V as fp16, two halves of 64 columns
constexpr int kHalfV = kTileV / 2;
constexpr int kStages = 2;               // code tiles in flight, K and V each
constexpr int kSoftmaxWarps = 8;
constexpr int kSoftmaxThreads = kSoftmaxWarps * 32;
constexpr int kThreads = 64 + kSoftmaxThreads;  // warp 0 TMA, warp 1 MMA, warps 2..9 softmax
constexpr int kCtasPerSm = 2;
constexpr int kSmemQ = 0;                            // hi, lo
constexpr int kSmemK = 2 * kTileQ;
constexpr int kSmemV8 = kSmemK + kStages * kTile8;
constexpr int kSmemV = kSmemV8 + kStages * kTile8;   // fp16 V of tile t at kSmemV + (t & 1) * kTileV
constexpr int kSmemBytes = kSmemV + 2 * kTileV;      // 96 KB
constexpr int kTmemCols = 256;  // S double buffer (2 x 64 columns; P over S), O (128)
constexpr uint32_t kTmemO = 128;
constexpr int kMaxW = kMaxSlots / 32;

// kind::f8f6f4, both operands e4m3 (type 0), fp32 accumulate; kind::f16 with both fp16 (type 0).
__host__ __device__ constexpr uint32_t idesc_type0(int M, int N, int b_mn_major) {
    return (1u << 4) | (static_cast<uint32_t>(b_mn_major) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void mma_f8(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, int accum) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(tmem_d),
        "l"(a), "l"(b), "r"(idesc), "r"(accum)
        : "memory");
}

__device__ __forceinline__ void named_sync_softmax() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory"); }
__device__ __forceinline__ void named_sync_pair(int q4) { asm volatile("bar.sync %0, 64;" ::"r"(2 + q4) : "memory"); }

__device__ __forceinline__ float max16(const float* v) {
    const float a = fmax3(v[0], v[1], v[2]), b = fmax3(v[3], v[4], v[5]), c = fmax3(v[6], v[7], v[8]);
    const float d = fmax3(v[9], v[10], v[11]), e = fmax3(v[12], v[13], v[14]);
    return fmaxf(fmax3(a, b, c), fmax3(d, e, v[15]));
}

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {  // a in the low byte
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(b), "f"(a));
    return d;
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    kvq_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, KvqAttnParams p) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t bar_q, bar_k_full[kStages], bar_k_empty[kStages], bar_v_full[kStages], bar_v_empty[kStages],
        bar_s_full[2], bar_p_full[2], bar_pv_done[2];
    __shared__ uint32_t tmem_holder;
    __shared__ float xch[2][2][kBM];  // [tile parity][column half][row]: per-tile row maxima
    __shared__ float lsum[2][kBM];    // [column half][row]: row sums of a piece

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int worker = blockIdx.x;
    if (threadIdx.x == 0) {
        mbar_init(&bar_q, kSoftmaxThreads);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bar_k_full[s], 1);
            mbar_init(&bar_k_empty[s], 1);
            mbar_init(&bar_v_full[s], 1);
            mbar_init(&bar_v_empty[s], kSoftmaxWarps);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar_s_full[s], 1);
            mbar_init(&bar_p_full[s], kSoftmaxThreads);
            mbar_init(&bar_pv_done[s], 1);
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_holder)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait_prior();
    pdl_launch_dependents();  // after the wait: the merge reads the lengths before its own
    KvqCursor cur;
    cur.init(p.s, worker);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_holder;
    const uint32_t tmem_s = tmem;           // S(t) at tmem_s + 64 (t & 1); P(t) over its first 32 columns
    const uint32_t tmem_o = tmem + kTmemO;  // O
    uint32_t* mask_sm = reinterpret_cast<uint32_t*>(smem + kSmemBytes);  // [row][W]: mask words of each row's slot
    KvqPiece it;

    if (warp == 0) {
        // ------------------------------------------------ TMA producers ---
        // Lane 0 loads the K tiles (a stage is free once QK^T of its tile is
        // done), lane 1 the V tiles (free once converted).
        if (lane < 2) {
            const bool is_k = lane == 0;
            uint64_t* full = is_k ? bar_k_full : bar_v_full;
            uint64_t* empty = is_k ? bar_k_empty : bar_v_empty;
            const CUtensorMap* map = is_k ? &tm_k : &tm_v;
            int t = 0;
            bool ok = true;
            while (ok && cur.next(p.s, it)) {
                const int hk = it.sub / p.n_rb;
                for (int j = it.t0; j < it.t1; ++j, ++t) {
                    const int st = t % kStages;
                    if (t >= kStages && !mbar_wait_sleep(&empty[st], ((t / kStages) - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&full[st], kTile8);
                    tma_load_4d(smem + (is_k ? kSmemK : kSmemV8) + st * kTile8, map, 0, hk, j * kBN, it.b, &full[st]);
                }
            }
            // the copies in flight land before the CTA's shared memory goes away
            if (!ok) {
                raise_status(p.status, kDevTimeout);
                for (int f = t > kStages ? t - kStages : 0; f < t; ++f)
                    mbar_wait_sleep(&full[f % kStages], (f / kStages) & 1, 1u << 10);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer ---
        // Tiles are numbered t over all of the worker's pieces. QK(t) goes
        // into S buffer t & 1, whose previous content P(t-2) was read by
        // PV(t-2), issued earlier (tcgen05.mma of one thread execute in issue
        // order). Issue order QK(0) QK(1) PV(0) QK(2) PV(1) ... A piece's
        // first PV overwrites O: the softmax threads have read the previous
        // piece's O before they arrive for it.
        if (lane == 0) {
            constexpr uint32_t id_qk = idesc_type0(kBM, kBN, 0);
            constexpr uint32_t id_pv = idesc_type0(kBM, kHD, 1);
            const uint32_t aQ = smem_u32(smem + kSmemQ);
            int t = 0, qi = 0;
            bool ok = true;
            auto issue_pv = [&](int tp, bool first) -> bool {
                const int sb = tp & 1;
                if (!mbar_wait_sleep(&bar_p_full[sb], (tp >> 1) & 1)) return false;  // P written, V converted
                tc_fence_after();
                const uint32_t aV = smem_u32(smem + kSmemV + sb * kTileV);
#pragma unroll
                for (int kk = 0; kk < kBN / 16; ++kk)  // A = P from TMEM: 16 keys = 8 columns per MMA
                    mma_bf16_ts(tmem_o, tmem_s + sb * kBN + kk * 8, smem_desc(aV + kk * 2048, kHalfV, 1024), id_pv,
                                (!first || kk > 0) ? 1 : 0);
                mma_commit(&bar_pv_done[sb]);
                return true;
            };
            while (ok && cur.next(p.s, it)) {
                if (!mbar_wait_sleep(&bar_q, qi & 1)) {
                    ok = false;
                    break;
                }
                ++qi;
                for (int j = it.t0; ok && j < it.t1; ++j, ++t) {
                    const int sb = t & 1, sk = t % kStages;
                    ok = mbar_wait_sleep(&bar_k_full[sk], (t / kStages) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t aK = smem_u32(smem + kSmemK + sk * kTile8);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)  // hi (0..3), lo (4..7); 32 elements of the head dimension each
                        mma_f8(tmem_s + sb * kBN, smem_desc(aQ + (kk >> 2) * kTileQ + (kk & 3) * 32, 16, 1024),
                               smem_desc(aK + (kk & 3) * 32, 16, 1024), id_qk, kk > 0);
                    mma_commit(&bar_k_empty[sk]);
                    mma_commit(&bar_s_full[sb]);
                    if (j > it.t0) ok = issue_pv(t - 1, j == it.t0 + 1);
                }
                if (ok) ok = issue_pv(t - 1, it.t1 - it.t0 == 1);
            }
            if (!ok) raise_status(p.status, kDevTimeout);
        }
    } else {
        // ------------------------------------------------------ softmax ---
        // Warp w serves TMEM lane quarter w % 4 (rows 32 q4 ..) and key
        // columns 32 h .. 32 h + 31 of each tile, h the warp's column half;
        // the two threads of a row exchange row maxima through shared memory.
        const int sw = warp - 2;
        const int h = sw >> 2;            // column half
        const int q4 = warp & 3;
        const int r = (q4 << 5) | lane;   // row of the block = TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
        int t = 0;                        // tiles so far
        bool ok = true;
        kvq_zero_bad(p.s, p.Hq, p.out, p.status, worker, threadIdx.x - 64, kSoftmaxThreads);
        while (cur.next(p.s, it)) {
            const int hk = it.sub / p.n_rb, rb = it.sub - hk * p.n_rb;
            const int row = rb * kBM + r;  // row of the (sequence, KV head)
            const int i = row / p.G;       // its tree slot
            const bool row_live = i < p.s.T;
            // a lane quarter whose 32 rows are all past the problem's rows does no
            // arithmetic on S (it still takes part in every barrier and conversion)
            const bool quarter_live = rb * kBM + q4 * 32 < p.G * p.s.T;
            const size_t qrow = ((static_cast<size_t>(it.b) * p.s.T + i) * p.Hq + static_cast<size_t>(hk) * p.G +
                                 (row - i * p.G)) * kHD;
            // ---- q: this thread's 64 elements as two e4m3 parts ----
            float fac;  // a score in the log2 domain, without K's scale
            {
                const uint4* src = reinterpret_cast<const uint4*>(p.q + qrow + 64 * h);
                uint4 u[8];
                uint32_t mx = 0u;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    u[e] = row_live ? __ldg(src + e) : make_uint4(0u, 0u, 0u, 0u);
                    mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(u[e].x & 0x7fff7fffu, u[e].y & 0x7fff7fffu),
                                               __vmaxu2(u[e].z & 0x7fff7fffu, u[e].w & 0x7fff7fffu)));
                }
                xch[t & 1][h][r] = __uint_as_float(max(mx & 0xffffu, mx >> 16) << 16);
                named_sync_pair(q4);
                const float s = pow2_to(fmaxf(xch[t & 1][0][r], xch[t & 1][1][r]), 7);
                fac = p.scale_log2 / s;
#pragma unroll
                for (int c = 0; c < 4; ++c) {  // 16 elements: one 16-byte chunk of each part
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint4& v = u[2 * c + (e >> 1)];
                        const uint32_t w0 = (e & 1) ? v.z : v.x, w1 = (e & 1) ? v.w : v.y;
                        const float x[4] = {__uint_as_float(w0 << 16) * s, __uint_as_float(w0 & 0xffff0000u) * s,
                                            __uint_as_float(w1 << 16) * s, __uint_as_float(w1 & 0xffff0000u) * s};
                        const uint32_t h0 = e4m3x2(x[0], x[1]), h1 = e4m3x2(x[2], x[3]);
                        const uint32_t f0 = e4m3_to_f16x2(h0), f1 = e4m3_to_f16x2(h1);
                        const float2 b0 = __half22float2(*reinterpret_cast<const __half2*>(&f0));
                        const float2 b1 = __half22float2(*reinterpret_cast<const __half2*>(&f1));
                        hi[e] = h0 | (h1 << 16);
                        lo[e] = e4m3x2(x[0] - b0.x, x[1] - b0.y) | (e4m3x2(x[2] - b1.x, x[3] - b1.y) << 16);
                    }
                    unsigned char* dst = smem + kSmemQ + r * kHD + (((4 * h + c) ^ (r & 7)) << 4);
                    *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(dst + kTileQ) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                fence_proxy_async_smem();  // the MMA reads q through the async proxy
                mbar_arrive(&bar_q);
            }
            if (h == 0) {  // the row's mask words
#pragma unroll
                for (int w = 0; w < kMaxW; ++w) {
                    if (w >= p.W) break;
                    uint32_t m = 0u;
                    if (row_live) {
                        if (p.mask) m = __ldg(&p.mask[(static_cast<size_t>(it.b) * p.s.T + i) * p.W + w]);
                        else m = i >= 32 * w + 31 ? ~0u : i < 32 * w ? 0u : (2u << (i - 32 * w)) - 1u;
                    }
                    mask_sm[r * p.W + w] = m;
                }
            }
            named_sync_softmax();
            const uint32_t* mrow = mask_sm + r * p.W;
            const int L = it.L, n = it.n;
            const float* ks = p.k_scale + it.b * p.s_seq + hk;
            const float* vs = p.v_scale + it.b * p.s_seq + hk;
            const int last = (it.nkeys - 1) >> p.blk_shift;
            // K's scales of this thread's two 16-key groups, V's of the tile's four: read a
            // tile ahead and used only then (their latency is that of a miss)
            float kc[2], vc[4];
            auto scales = [&](int j) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    vc[e] = __ldg(vs + min((j * kBN + 16 * e) >> p.blk_shift, last) * p.s_blk);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    kc[e] = __ldg(ks + min((j * kBN + 32 * h + 16 * e) >> p.blk_shift, last) * p.s_blk);
            };
            scales(it.t0);
            float m_use = 0.0f, lh = 0.0f, sref = 0.0f;  // lh: this half's share of the row sum
            bool seen = false;
            for (int j = it.t0; j < it.t1; ++j, ++t) {
                const int sb = t & 1;
                const int key0 = j * kBN;
                const uint32_t s_cols = tmem_s + sb * kBN;
                const float k0 = kc[0] * fac, k1 = kc[1] * fac, v0 = h ? vc[2] : vc[0], v1 = h ? vc[3] : vc[1];
                const float vmax = fmaxf(fmaxf(vc[0], vc[1]), fmaxf(vc[2], vc[3]));
                if (j + 1 < it.t1) scales(j + 1);
                // ---- V of this tile: 16 columns of two keys per thread, codes to fp16 ----
                {
                    const int st = t % kStages;
                    if (ok && (!__all_sync(0xffffffffu, mbar_wait_sleep(&bar_v_full[st], (t / kStages) & 1)) ||
                               (t >= 2 && !__all_sync(0xffffffffu, mbar_wait_sleep(&bar_pv_done[sb], ((t >> 1) - 1) & 1)))))
                        ok = false;
                    if (ok) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int key = lane + 32 * e;
                            uint4 u = *reinterpret_cast<const uint4*>(smem + kSmemV8 + st * kTile8 + key * kHD +
                                                                      ((sw ^ (key & 7)) << 4));
                            // keys that no row can see may hold anything (even NaN): 0 * V has to stay 0
                            if (key0 + key >= it.nkeys) u = make_uint4(0u, 0u, 0u, 0u);
                            unsigned char* dst = smem + kSmemV + sb * kTileV + (sw >> 2) * kHalfV + key * 128;
                            const int c = 2 * (sw & 3);
                            *reinterpret_cast<uint4*>(dst + ((c ^ (key & 7)) << 4)) =
                                make_uint4(e4m3_to_f16x2(u.x & 0xffffu), e4m3_to_f16x2(u.x >> 16),
                                           e4m3_to_f16x2(u.y & 0xffffu), e4m3_to_f16x2(u.y >> 16));
                            *reinterpret_cast<uint4*>(dst + (((c + 1) ^ (key & 7)) << 4)) =
                                make_uint4(e4m3_to_f16x2(u.z & 0xffffu), e4m3_to_f16x2(u.z >> 16),
                                           e4m3_to_f16x2(u.w & 0xffffu), e4m3_to_f16x2(u.w >> 16));
                        }
                        fence_proxy_async_smem();  // the MMA reads V through the async proxy
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar_v_empty[st]);
                    }
                }
                // After a timed-out wait a warp skips the work of the remaining tiles
                // but still takes every named barrier, so the others never wait for
                // it without bound.
                if (ok && !__all_sync(0xffffffffu, mbar_wait_sleep(&bar_s_full[sb], (t >> 1) & 1))) ok = false;
                tc_fence_after();
                float sv[32];
                if (ok && quarter_live) {
                    tmem_ld32(s_cols + lane_off + 32 * h, sv);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) sv[e] = -INFINITY;
                }
                // visibility of the half's 32 keys: prefix keys, then tree slots in mask row i
                {
                    const int kb = key0 + 32 * h;
                    const int npre = L - kb;  // keys of the 32 inside the prefix
                    if (npre < 32) {
                        const uint32_t pre = npre > 0 ? (1u << npre) - 1u : 0u;
                        const int j0 = kb - L;  // slot of the first key (may be negative)
                        const int lo = j0 < 0 ? 0 : j0;
                        const int w0 = lo >> 5, sh = lo & 31;
                        uint32_t win = w0 < p.W ? mrow[w0] >> sh : 0u;
                        if (sh && w0 + 1 < p.W) win |= mrow[w0 + 1] << (32 - sh);
                        const int limit = n - lo;  // slots j >= n are never visible
                        if (limit <= 0) win = 0u;
                        else if (limit < 32) win &= (1u << limit) - 1u;
                        uint32_t tree = j0 < 0 ? (win << (-j0 & 31)) : win;
                        if (j0 <= -32) tree = 0u;
                        const uint32_t vis = pre | tree;
#pragma unroll
                        for (int e = 0; e < 32; ++e) sv[e] = ((vis >> e) & 1u) ? sv[e] : -INFINITY;
                    }
                }
                float mx = fmaxf(max16(sv) * k0, max16(sv + 16) * k1);  // the scales are positive
                if (quarter_live) {
                    xch[t & 1][h][r] = mx;
                    tc_fence_before();
                    named_sync_pair(q4);  // also: both halves have read S, so P may overwrite it
                    tc_fence_after();
                    mx = fmaxf(xch[t & 1][0][r], xch[t & 1][1][r]);
                }
                bool rescale = false;
                float alpha = 1.0f;
                if (mx > -INFINITY) {
                    if (!seen) {
                        m_use = mx;  // O and l are still zero for this piece
                        seen = true;
                    } else if (mx > m_use + 8.0f) {
                        alpha = ex2_approx(m_use - mx);
                        m_use = mx;
                        rescale = true;
                        lh *= alpha;
                    }
                }
                if (vmax > 16.0f * sref) {  // uniform: the tile's largest V scale
                    alpha *= sref / vmax;
                    rescale = sref > 0.0f;
                    sref = vmax;
                }
                if (!ok) continue;
                if (quarter_live) {
                    // p = 2^(s k - m_use), two per packed multiply-add; packed partial sums.
                    // P(t) as fp16 pairs over S columns 16 h .. 16 h + 15 of this buffer.
                    const uint64_t nm2 = f2_pack(-m_use, -m_use);
                    const float rs = 1.0f / sref;
                    uint64_t acc[2] = {0ull, 0ull};
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float kk = e < 16 ? k0 : k1, vv = (e < 16 ? v0 : v1) * rs;
                        const uint64_t z = f2_fma(f2_pack(sv[e], sv[e + 1]), f2_pack(kk, kk), nm2);
                        const uint64_t w = f2_pack(ex2_approx(f2_lo(z)), ex2_approx(f2_hi(z)));
                        acc[(e >> 1) & 1] = f2_add(acc[(e >> 1) & 1], w);
                        const uint64_t x = f2_mul(w, f2_pack(vv, vv));
                        pk[e >> 1] = pack_f16(f2_lo(x), f2_hi(x));
                    }
                    tmem_st16(s_cols + lane_off + 16 * h, pk);
                    const uint64_t s2 = f2_add(acc[0], acc[1]);
                    lh += f2_lo(s2) + f2_hi(s2);
                }
                // Rescaling O needs PV(t-1) done (PV(t) waits for this thread's
                // arrival below). tcgen05.ld/st are warp-collective: rescale if any
                // row of the warp needs it (alpha = 1 for the others).
                if (quarter_live && j > it.t0 && __any_sync(0xffffffffu, rescale)) {
                    if (!__all_sync(0xffffffffu, mbar_wait_sleep(&bar_pv_done[sb ^ 1], ((t - 1) >> 1) & 1))) {
                        ok = false;
                    } else {
                        tc_fence_after();
#pragma unroll
                        for (int hq = 0; hq < 2; ++hq) {
                            float o[32];
                            tmem_ld32(tmem_o + lane_off + 64 * h + 32 * hq, o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= alpha;
                            tmem_st32(tmem_o + lane_off + 64 * h + 32 * hq, o);
                        }
                    }
                }
                tc_fence_before();
                mbar_arrive(&bar_p_full[sb]);
            }
            // the piece's last PV done: O final, q and the V buffers free
            if (ok && !__all_sync(0xffffffffu, mbar_wait_sleep(&bar_pv_done[(t - 1) & 1], ((t - 1) >> 1) & 1))) ok = false;
            if (!ok) raise_status(p.status, kDevTimeout);
            // ----------------------------------------------------- epilogue ---
            // Thread (row r, half h) owns output columns 64 h .. 64 h + 63 of its row.
            lsum[h][r] = lh;
            named_sync_softmax();  // row sums of both halves; every mask row has been read
            tc_fence_after();
            const float l = lsum[0][r] + lsum[1][r];
            const bool any = row_live && quarter_live && seen && l > 0.0f && ok;
            if (it.whole()) {
                const bool live = any && i < n;  // unused slots: zeros
                const float inv = live ? sref / l : 0.0f;
                __nv_bfloat16* orow = p.out + qrow + 64 * h;
#pragma unroll
                for (int hq = 0; hq < 2; ++hq) {
                    float o[32];
                    tmem_ld32(tmem_o + lane_off + 64 * h + 32 * hq, o);
                    if (!row_live) continue;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint4 uo = make_uint4(0u, 0u, 0u, 0u);
                        if (live)
                            uo = make_uint4(pack_bf16(o[8 * q] * inv, o[8 * q + 1] * inv),
                                            pack_bf16(o[8 * q + 2] * inv, o[8 * q + 3] * inv),
                                            pack_bf16(o[8 * q + 4] * inv, o[8 * q + 5] * inv),
                                            pack_bf16(o[8 * q + 6] * inv, o[8 * q + 7] * inv));
                        *reinterpret_cast<uint4*>(orow + 32 * hq + 8 * q) = uo;
                    }
                }
            } else {
                const size_t at = static_cast<size_t>(it.slot(worker)) * kBM + r;
                float* po = p.part.o + at * kHD + 64 * h;
#pragma unroll
                for (int hq = 0; hq < 2; ++hq) {
                    float o[32];
                    tmem_ld32(tmem_o + lane_off + 64 * h + 32 * hq, o);
                    if (!row_live) continue;
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        *reinterpret_cast<float4*>(po + 32 * hq + 4 * q) =
                            any ? make_float4(o[4 * q] * sref, o[4 * q + 1] * sref, o[4 * q + 2] * sref, o[4 * q + 3] * sref)
                                : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
                if (row_live && h == 0) {
                    p.part.ml[2 * at] = any ? m_use : -INFINITY;
                    p.part.ml[2 * at + 1] = any ? l : 0.0f;
                }
            }
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// ------------------------------------------------------------- host side ---

struct Plan {
    KvqSched s;
    int G, n_rb, rows;
    bool decode;
    size_t off_ml, off_o, bytes;
};

// Up to 16 query rows per KV head: the decode kernel, a worker per warp;
// more: the tensor-core kernel, a worker per CTA. A rule on rows because the
// first keeps 16 x 128 sums in a warp's registers.
Plan make_plan(const KvqDims& kv, int T) {
    Plan pl{};
    pl.G = kv.Hq / kv.Hkv;
    pl.decode = static_cast<long>(pl.G) * T <= kKvqDecodeRows;
    if (pl.decode) {
        pl.n_rb = 1;
        pl.rows = pl.G * T;
        pl.s = kvq_decode_sched(kv.B, T, kv.max_len, kv.Hkv);
    } else {
        pl.n_rb = (pl.G * T + kBM - 1) / kBM;
        pl.rows = kBM;
        pl.s = KvqSched{nullptr, nullptr, kv.B, T, kv.max_len, kv.Hkv * pl.n_rb, kBN, 3, kKvqSms * kCtasPerSm, 6};
    }
    const size_t slots = 2 * static_cast<size_t>(pl.s.workers) * pl.rows;
    pl.off_ml = 256;
    pl.off_o = align_up(pl.off_ml + slots * 2 * sizeof(float), 256);
    pl.bytes = align_up(pl.off_o + slots * kHD * sizeof(float), 256);
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
    p.part = KvqPartials{reinterpret_cast<float*>(w + pl.off_o), reinterpret_cast<float*>(w + pl.off_ml), pl.rows};
    p.Hq = kv.Hq;
    p.Hkv = kv.Hkv;
    p.G = pl.G;
    p.n_rb = pl.n_rb;
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
    cudaError_t e;
    if (pl.decode) {
        e = launch_kvq_decode(kv, p, kbase, vbase, stream);
    } else {
        CUtensorMap tk, tv;
        if (!make_map_codes(&tk, kbase, kv, kBN) || !make_map_codes(&tv, vbase, kv, kBN)) return cudaErrorInvalidValue;
        const int dyn = kSmemBytes + kBM * p.W * 4 + 1024;  // stages, mask rows, alignment slack
        e = ensure_dyn_smem(reinterpret_cast<const void*>(kvq_attn_kernel), dyn);
        if (e != cudaSuccess) return e;
        static std::once_flag carve;  // two CTAs per SM need the largest shared-memory carveout
        std::call_once(carve, [] {
            cudaFuncSetAttribute(reinterpret_cast<const void*>(kvq_attn_kernel),
                                 cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        });
        e = launch_pdl(kvq_attn_kernel, dim3(pl.s.workers), dim3(kThreads), dyn, stream, tk, tv, p);
    }
    if (e != cudaSuccess) return e;
    return launch_kvq_merge(KvqMergeParams{pl.s, p.part, p.G, T, p.Hq, p.n_rb, p.out}, stream);
}

}  // namespace eagle
