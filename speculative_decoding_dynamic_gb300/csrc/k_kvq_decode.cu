// Attention over the 8-bit KV cache for few query rows (sm_103a): G * T <= 16
// rows per KV head (decode steps, chains and small trees).
//
// out = softmax(q k^T) v with k, v = code * scale of a block. Every key is used
// by at most 16 rows, so reading the cache is the cost: 2 * 128 bytes per key
// and head, 32 flops a byte at 4 rows, far below the tensor cores' ridge.
// The kernel keeps many bytes in flight and does little per byte:
//   - a warp is a worker of the split (kvq_sched.cuh) and works alone: it
//     streams its keys 32 at a time through its own ring of TMA tiles
//     (4 KB of K, 4 KB of V a stage) and keeps the running maximum, sum and
//     accumulator in registers. No barrier between warps.
//   - the products run transposed, S^T = K q^T and O^T = V^T P^T, on mma.sync
//     m16n8k16 with the cache as the 16-row operand: eight query rows are one
//     n-tile (with q as the 16-row operand twelve of its rows would be empty
//     for a group of four heads). tcgen05's
//     128-row tile would need the operands as fp16 in shared memory, twice
//     their bytes written and read again.
//   - codes go from shared memory to fp16 fragments by one conversion per two
//     elements (exact); P^T is turned around in registers (movmatrix).
//   - q is scaled per row by a power of two into fp16's range (exact but for
//     elements below 2^-28 of the row's largest).
//   - K's scale multiplies the scores; V's multiplies the softmax weights,
//     relative to a reference scale that is raised like the maximum.
// Measured: 64 sequences of 256..2048 positions, 8B heads (152 MB of cache):
// 40.8 us with the merge (some 5 us) in a captured graph, 41 to 43 call after
// call; the kernel reads at 4.2 TB/s.
// Fragment layouts: the head dimension is summed over in an order in which
// lane t of a quad holds bytes 16t..16t+15 and 64+16t.. of a K row (two 16-byte
// loads), and the output columns are taken in an order in which a lane holds 16
// neighbouring columns of a V row (one 16-byte load per key).

#include "kvq_sched.cuh"

namespace eagle {
namespace {

constexpr int kStep = 32;                      // keys per stage
constexpr int kTile = kStep * kKvqHeadDim;     // 4 KB
constexpr int kStageBytes = 2 * kTile;
// Up to eight rows: twelve warps of two stages; up to sixteen (twice the
// accumulators): eight of three. 192 KB of ring either way.
constexpr int warps_of(int NT) { return NT == 1 ? 12 : 8; }
constexpr int stages_of(int NT) { return NT == 1 ? 2 : 3; }
constexpr int kSmem = 192 * 1024 + 1024;

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit elements held two per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// 16 bf16 as fp16, scaled by a power of two.
__device__ __forceinline__ void q_to_f16(const uint4& u, float s, uint32_t* d) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        d[i] = pack_f16(__uint_as_float(w[i] << 16) * s, __uint_as_float(w[i] & 0xffff0000u) * s);
}
__device__ __forceinline__ float absmax8(const uint4& u) {
    const uint32_t m = __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu),
                                __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
    return __uint_as_float(max(m & 0xffffu, m >> 16) << 16);
}

template <int NT>
__global__ void __launch_bounds__(warps_of(NT) * 32, 1)
    kvq_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      KvqAttnParams p) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    constexpr int kStages = stages_of(NT);
    __shared__ uint64_t bar[warps_of(NT)][kStages];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int worker = warp * gridDim.x + blockIdx.x;  // neighbouring workers on different SMs
    const int g = lane >> 2, t = lane & 3;
    unsigned char* ring = smem + warp * kStages * kStageBytes;
    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(&bar[warp][s], 1);
        fence_mbar_init();
    }
    __syncwarp();
    pdl_wait_prior();
    pdl_launch_dependents();
    kvq_zero_bad(p.s, p.Hq, p.out, p.status, worker, lane, 32);

    KvqCursor cur, ahead;
    cur.init(p.s, worker);
    ahead = cur;
    KvqPiece np;  // the piece that the ring is being filled from
    bool more = ahead.next(p.s, np);
    int nt_at = more ? np.t0 : 0;
    int filled = 0, used = 0;
    auto fill = [&]() {  // the next step's tiles into the ring
        if (!more) return;
        const int s = filled % kStages;
        if (lane == 0) {
            uint64_t* b = &bar[warp][s];
            mbar_arrive_expect_tx(b, kStageBytes);
            tma_load_4d(ring + s * kStageBytes, &tm_k, 0, np.sub, nt_at * kStep, np.b, b);
            tma_load_4d(ring + s * kStageBytes + kTile, &tm_v, 0, np.sub, nt_at * kStep, np.b, b);
        }
        ++filled;
        if (++nt_at == np.t1) {
            more = ahead.next(p.s, np);
            nt_at = more ? np.t0 : 0;
        }
    };
#pragma unroll
    for (int s = 0; s < kStages; ++s) fill();

    const int rows = p.G * p.s.T;
    bool ok = true;
    int4 cut = make_int4(0, 0, 0, 0);
    KvqPiece it;
    while (cur.next(p.s, it)) {
        if (it.np) cut = kvq_cut(it);
        const int hk = it.sub;
        // q rows 8 nt + g as B fragments; a score of row 8 nt + 2t + e to the log2 domain; that row's
        // visible tree slots (T <= 16: one mask word)
        uint32_t qb[NT][8][2];
        float fac[NT][2];
        uint32_t see[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = 8 * nt + g;
            const int slot = r / p.G;
            uint4 u[4] = {};
            uint32_t vis = 0u;
            if (r < rows) {
                const uint4* src = reinterpret_cast<const uint4*>(
                    p.q + ((static_cast<size_t>(it.b) * p.s.T + slot) * p.Hq + hk * p.G + (r - slot * p.G)) * kKvqHeadDim);
                u[0] = ld_prior(src + 2 * t);
                u[1] = ld_prior(src + 2 * t + 1);
                u[2] = ld_prior(src + 8 + 2 * t);
                u[3] = ld_prior(src + 8 + 2 * t + 1);
                vis = p.mask ? ld_prior(&p.mask[static_cast<size_t>(it.b) * p.s.T + slot]) : (2u << slot) - 1u;
                vis &= (1u << it.n) - 1u;  // n <= 16
            }
            float am = fmaxf(fmaxf(absmax8(u[0]), absmax8(u[1])), fmaxf(absmax8(u[2]), absmax8(u[3])));
            am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
            am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
            const float s = pow2_to(am, 14);
            uint32_t d[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) q_to_f16(u[i], s, d + 4 * i);
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // MMA i sums over bytes 4i..4i+3 of the lane's 32
                qb[nt][i][0] = d[2 * i];
                qb[nt][i][1] = d[2 * i + 1];
            }
            const float f = p.scale_log2 / s;
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // row 2t + e is held by the lanes 4 (2t + e) ..
                fac[nt][e] = __shfl_sync(0xffffffffu, f, 4 * (2 * t + e));
                see[nt][e] = __shfl_sync(0xffffffffu, vis, 4 * (2 * t + e));
            }
        }
        float o[NT][8][4];  // columns 16 g + 2j (+ 1: [2], [3]) of rows 8 nt + 2t ([0], [2]) and 2t + 1
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.0f;
        }
        float sref = 0.0f, inv_sref = 0.0f;
        // scales of a step's two 16-key halves, read a step ahead
        const float* ks = p.k_scale + it.b * p.s_seq + hk;
        const float* vs = p.v_scale + it.b * p.s_seq + hk;
        const int last = (it.nkeys - 1) >> p.blk_shift;
        float kc[2], vc[2];
        auto scales = [&](int step) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int64_t at = min((step * kStep + 16 * e) >> p.blk_shift, last) * p.s_blk;
                kc[e] = ld_prior(ks + at);
                vc[e] = ld_prior(vs + at);
            }
        };
        scales(it.t0);
        for (int step = it.t0; step < it.t1; ++step) {
            const int st = used % kStages;
            const uint32_t sk = smem_u32(ring) + st * kStageBytes, sv = sk + kTile;
            const int key0 = step * kStep;
            const float kk[2] = {kc[0], kc[1]}, vv[2] = {vc[0], vc[1]};
            if (step + 1 < it.t1) scales(step + 1);
            if (ok && !__all_sync(0xffffffffu, mbar_wait(&bar[warp][st], (used / kStages) & 1))) {
                // a copy that never landed: no more reading, nothing is refilled,
                // and the other copies land before shared memory goes away
                ok = false;
                if (lane == 0) raise_status(p.status, kDevTimeout);
                for (int f = used + 1; f < filled; ++f) mbar_wait(&bar[warp][f % kStages], (f / kStages) & 1);
            }
            ++used;
            if (!ok) continue;
            // ---- scores: keys 16 hf + g ([0], [1]) and + 8; rows 8 nt + 2t, + 1 ----
            float s[2][NT][4];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) s[hf][nt][0] = s[hf][nt][1] = s[hf][nt][2] = s[hf][nt][3] = 0.0f;
                const uint32_t row = sk + (hf * 16 + g) * kKvqHeadDim;  // the swizzle of keys g and g + 8 is the same
                const uint4 a = lds128(row + ((t ^ g) << 4)), b = lds128(row + (((t + 4) ^ g) << 4));
                const uint4 c = lds128(row + 8 * kKvqHeadDim + ((t ^ g) << 4));
                const uint4 d = lds128(row + 8 * kKvqHeadDim + (((t + 4) ^ g) << 4));
                const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                const uint32_t x[8] = {c.x, c.y, c.z, c.w, d.x, d.y, d.z, d.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t a0 = e4m3_to_f16x2(w[i]), a1 = e4m3_to_f16x2(x[i]);
                    const uint32_t a2 = e4m3_to_f16x2(w[i] >> 16), a3 = e4m3_to_f16x2(x[i] >> 16);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16(s[hf][nt], a0, a1, a2, a3, qb[nt][i][0], qb[nt][i][1]);
                }
            }
            // ---- log2 domain, tree mask, maxima ----
            float mx[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[hf][nt][e] *= kk[hf] * fac[nt][e & 1];
                if (key0 + kStep > it.L) {
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = key0 + hf * 16 + g + 8 * (e >> 1) - it.L;  // tree slot (< 0: prefix)
                            if (j >= 0 && !(j < 32 && ((see[nt][e & 1] >> j) & 1u))) s[hf][nt][e] = -INFINITY;
                        }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = fmaxf(fmaxf(s[0][nt][e], s[0][nt][e + 2]), fmaxf(s[1][nt][e], s[1][nt][e + 2]));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                    mx[nt][e] = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                }
            }
            // ---- running maximum and reference V scale, raised only by more than 2^8 (2^4): weights stay below 2^12 ----
            float al[NT][2];
            bool raise = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    al[nt][e] = 1.0f;
                    if (mx[nt][e] > m[nt][e] + 8.0f) {  // -inf at first
                        al[nt][e] = m[nt][e] == -INFINITY ? 0.0f : ex2_approx(m[nt][e] - mx[nt][e]);
                        m[nt][e] = mx[nt][e];
                        l[nt][e] *= al[nt][e];
                        raise = true;
                    }
                }
            const float vm = fmaxf(fmaxf(vv[0], vv[1]), kKvqMinRef);
            if (vm > 16.0f * sref) {  // uniform over the warp
                const float r = sref / vm;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    al[nt][0] *= r;
                    al[nt][1] *= r;
                }
                sref = vm;
                inv_sref = 1.0f / vm;
                raise = true;
            }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[nt][j][e] *= al[nt][e & 1];
            }
            // ---- weights, transposed into B fragments ----
            uint32_t pb[2][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float mu[2] = {m[nt][0] == -INFINITY ? 0.0f : m[nt][0], m[nt][1] == -INFINITY ? 0.0f : m[nt][1]};
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const float rv = vv[hf] * inv_sref;
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        w[e] = ex2_approx(s[hf][nt][e] - mu[e & 1]);
                        l[nt][e & 1] += w[e];
                    }
                    pb[hf][nt][0] = transpose8(pack_f16(w[0] * rv, w[1] * rv));
                    pb[hf][nt][1] = transpose8(pack_f16(w[2] * rv, w[3] * rv));
                }
            }
            // ---- O += P V: keys 16 hf + {2t, 2t+1, 8+2t, 8+2t+1}, columns 16 g .. 16 g + 15 ----
            const bool tail = key0 + kStep > it.nkeys;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                uint4 u[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = hf * 16 + (e >> 1) * 8 + 2 * t + (e & 1);
                    u[e] = lds128(sv + key * kKvqHeadDim + ((g ^ (key & 7)) << 4));
                    if (tail && key0 + key >= it.nkeys) u[e] = make_uint4(0u, 0u, 0u, 0u);  // unwritten: may be NaN
                }
                const uint32_t w[4][4] = {{u[0].x, u[0].y, u[0].z, u[0].w},
                                          {u[1].x, u[1].y, u[1].z, u[1].w},
                                          {u[2].x, u[2].y, u[2].z, u[2].w},
                                          {u[3].x, u[3].y, u[3].z, u[3].w}};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a = __byte_perm(w[0][i], w[1][i], 0x5140), b = __byte_perm(w[2][i], w[3][i], 0x5140);
                    const uint32_t c = __byte_perm(w[0][i], w[1][i], 0x7362), d = __byte_perm(w[2][i], w[3][i], 0x7362);
                    const uint32_t a0 = e4m3_to_f16x2(a), a1 = e4m3_to_f16x2(a >> 16), a2 = e4m3_to_f16x2(b), a3 = e4m3_to_f16x2(b >> 16);
                    const uint32_t c0 = e4m3_to_f16x2(c), c1 = e4m3_to_f16x2(c >> 16), c2 = e4m3_to_f16x2(d), c3 = e4m3_to_f16x2(d >> 16);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_f16(o[nt][2 * i], a0, a1, a2, a3, pb[hf][nt][0], pb[hf][nt][1]);
                        mma_f16(o[nt][2 * i + 1], c0, c1, c2, c3, pb[hf][nt][0], pb[hf][nt][1]);
                    }
                }
            }
            __syncwarp();  // every lane has read the stage
            fill();
        }
        // ---- the piece's rows: columns 16g .. 16g+15 of rows 8 nt + 2t, + 1 ----
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[nt][e];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                const int r = 8 * nt + 2 * t + e;
                if (r >= rows) continue;
                float x[16];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[2 * j] = o[nt][j][e];
                    x[2 * j + 1] = o[nt][j][2 + e];
                }
                if (it.whole()) {
                    const int slot = r / p.G;
                    const bool live = ok && slot < it.n && sum > 0.0f;
                    const float inv = live ? sref / sum : 0.0f;
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = live ? pack_bf16(x[2 * i] * inv, x[2 * i + 1] * inv) : 0u;
                    uint4* dst = reinterpret_cast<uint4*>(
                        p.out + ((static_cast<size_t>(it.b) * p.s.T + slot) * p.Hq + hk * p.G + (r - slot * p.G)) * kKvqHeadDim +
                        16 * g);
                    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
                } else {
                    const size_t row = static_cast<size_t>(it.slot(worker)) * p.part.rows + r;
                    float4* dst = reinterpret_cast<float4*>(p.part.o + row * kKvqHeadDim + 16 * g);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        dst[c] = make_float4(x[4 * c] * sref, x[4 * c + 1] * sref, x[4 * c + 2] * sref, x[4 * c + 3] * sref);
                    if (g == 0) {
                        p.part.ml[2 * row] = ok ? m[nt][e] : -INFINITY;
                        p.part.ml[2 * row + 1] = ok ? sum : 0.0f;
                    }
                }
            }
    }
    if (lane == 0) p.part.cut[worker] = cut;
}

// ------------------------------------------------------------------ merge ---

constexpr int kMergeWarps = 8;
constexpr int kMergeAlone = 4;  // most pieces that one warp combines by itself

// Running combination of a row's pieces, four columns per lane.
// c: (pieces, sequence, item, tree size) of a cut item.
__device__ __forceinline__ void merge_store(const KvqMergeParams& p, const int4& c, int r, const RowSum<1>& s, int lane) {
    int slot;
    const int64_t row = p.rows.row(c.y, c.z, r, &slot);  // an item is a KV head
    if (row < 0) return;
    const bool live = slot < c.w && s.l > 0.0f;
    const float inv = live ? 1.0f / s.l : 0.0f;
    uint2* dst = reinterpret_cast<uint2*>(p.out + row * kKvqHeadDim);
    dst[lane] = live ? make_uint2(pack_bf16(s.o[0].x * inv, s.o[0].y * inv), pack_bf16(s.o[0].z * inv, s.o[0].w * inv))
                     : make_uint2(0u, 0u);
}

// The cut item that worker w began: O = sum_i 2^(m_i - M) O_i over
// sum_i 2^(m_i - M) l_i of its pieces i (worker w's in slot 2w + 1, w + i's in
// slot 2 (w + i)). A CTA serves the items that eight neighbouring workers
// began, one row of them (blockIdx.y): those of up to four pieces go to one
// warp each, those of many (few long sequences) are shared by all eight warps.
__global__ void __launch_bounds__(kMergeWarps * 32) kvq_merge_decode_kernel(KvqMergeParams p) {
    __shared__ float4 so[kMergeWarps][32];
    __shared__ float2 sml[kMergeWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int w0 = blockIdx.x * kMergeWarps, r = blockIdx.y;
    pdl_wait_prior();
    pdl_launch_dependents();
    const int4* items = p.part.cut + w0;
    const int n_here = min(kMergeWarps, p.workers - w0);
    const float2* ml = reinterpret_cast<const float2*>(p.part.ml);
    const float4* po = reinterpret_cast<const float4*>(p.part.o);
    auto slot_row = [&](int w, int i, int r) {
        return static_cast<size_t>(i == 0 ? 2 * w + 1 : 2 * (w + i)) * p.part.rows + r;
    };
    const int4 own = __ldcg(items + min(warp, n_here - 1));
    if (warp < n_here && own.x > 0 && own.x <= kMergeAlone) {
        RowSum<1> s;
        float2 a[kMergeAlone];
        float4 x[kMergeAlone][1];
#pragma unroll
        for (int i = 0; i < kMergeAlone; ++i) {
            if (i >= own.x) break;
            const size_t at = slot_row(w0 + warp, i, r);
            a[i] = __ldcg(ml + at);
            x[i][0] = __ldcg(po + at * 32 + lane);
        }
#pragma unroll
        for (int i = 0; i < kMergeAlone; ++i)
            if (i < own.x) s.add(a[i].x, a[i].y, x[i]);
        merge_store(p, own, r, s, lane);
    }
    for (int e = 0; e < n_here; ++e) {
        const int4 c = __ldcg(items + e);
        if (c.x <= kMergeAlone) continue;  // uniform over the CTA
        RowSum<1> s;
#pragma unroll 4
        for (int i = warp; i < c.x; i += kMergeWarps) {
            const size_t at = slot_row(w0 + e, i, r);
            const float2 a = __ldcg(ml + at);
            const float4 x[1] = {__ldcg(po + at * 32 + lane)};
            s.add(a.x, a.y, x);
        }
        so[warp][lane] = s.o[0];
        if (lane == 0) sml[warp] = make_float2(s.m, s.l);
        __syncthreads();
        if (warp == 0) {
            for (int i = 1; i < kMergeWarps; ++i) {
                const float4 x[1] = {so[i][lane]};
                s.add(sml[i].x, sml[i].y, x);
            }
            merge_store(p, c, r, s, lane);
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_kvq_merge_decode(const KvqMergeParams& p, cudaStream_t stream) {
    return launch_pdl(kvq_merge_decode_kernel, dim3((p.workers + kMergeWarps - 1) / kMergeWarps, p.part.rows), dim3(kMergeWarps * 32),
                      0, stream, p);
}

KvqSched kvq_decode_sched(int B, int T, int max_len, int Hkv, int rows) {
    return KvqSched{nullptr, nullptr, B, T, max_len, Hkv, 1, kStep, 2, 1, 1, kKvqSms * warps_of(rows <= 8 ? 1 : 2), 4};
}

template <int NT>
static cudaError_t launch_decode(const KvqAttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t stream) {
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kvq_decode_kernel<NT>), kSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kvq_decode_kernel<NT>, dim3(kKvqSms), dim3(warps_of(NT) * 32), kSmem, stream, tk, tv, p);
}

cudaError_t launch_kvq_decode(const KvqDims& kv, const KvqAttnParams& p, const void* kbase, const void* vbase,
                              cudaStream_t stream) {
    CUtensorMap tk, tv;
    if (!make_map_codes(&tk, kbase, kv, kStep) || !make_map_codes(&tv, vbase, kv, kStep)) return cudaErrorInvalidValue;
    return p.G * p.s.T <= 8 ? launch_decode<1>(p, tk, tv, stream) : launch_decode<2>(p, tk, tv, stream);
}

}  // namespace eagle
