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
//     the 16 x 128 accumulator in registers. No barrier between warps.
//   - codes go from shared memory to fp16 fragments by one conversion per two
//     elements (exact), and the products run on mma.sync m16n8k16: with at most
//     16 rows the tcgen05 tile (128 rows) would be seven eighths empty, and the
//     operands would have to be written back to shared memory as fp16.
//   - q is scaled per row by a power of two into fp16's range (exact but for
//     elements below 2^-28 of the row's largest).
//   - K's scale multiplies the scores; V's multiplies the softmax weights,
//     relative to a reference scale that is raised like the maximum.
// Fragment layouts: the head dimension is summed over in an order in which
// lane t of a quad holds bytes 16t..16t+15 and 64+16t.. of a K row (two 16-byte
// loads), and the output columns are taken in an order in which a lane holds 16
// neighbouring columns of a V row (one 16-byte load per key).

#include "kvq_sched.cuh"

namespace eagle {
namespace {

constexpr int kStep = 32;                      // keys per stage
constexpr int kStages = 3;
constexpr int kWarps = 8;                      // workers per CTA, one CTA per SM
constexpr int kTile = kStep * kKvqHeadDim;     // 4 KB
constexpr int kStageBytes = 2 * kTile;
constexpr int kSmem = kWarps * kStages * kStageBytes + 1024;

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

__global__ void __launch_bounds__(kWarps * 32, 1)
    kvq_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      KvqAttnParams p) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t bar[kWarps][kStages];
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
    pdl_launch_dependents();  // after the wait: the merge reads the lengths before its own
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
    KvqPiece it;
    while (cur.next(p.s, it)) {
        const int hk = it.sub;
        // q of rows g and g + 8 as A fragments, and the factor that takes a score to the log2 domain
        uint32_t qa[8][4];
        float fac[2];
        uint32_t see[2];  // visible tree slots of the row's slot (T <= 16: one mask word)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = g + 8 * e;
            const int slot = r / p.G;
            uint4 u[4] = {};
            see[e] = 0u;
            if (r < rows) {
                const uint4* src = reinterpret_cast<const uint4*>(
                    p.q + ((static_cast<size_t>(it.b) * p.s.T + slot) * p.Hq + hk * p.G + (r - slot * p.G)) * kKvqHeadDim);
                u[0] = __ldg(src + 2 * t);
                u[1] = __ldg(src + 2 * t + 1);
                u[2] = __ldg(src + 8 + 2 * t);
                u[3] = __ldg(src + 8 + 2 * t + 1);
                see[e] = p.mask ? __ldg(&p.mask[static_cast<size_t>(it.b) * p.s.T + slot]) : (2u << slot) - 1u;
                see[e] &= (1u << it.n) - 1u;  // n <= 16
            }
            float am = fmaxf(fmaxf(absmax8(u[0]), absmax8(u[1])), fmaxf(absmax8(u[2]), absmax8(u[3])));
            am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
            am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
            const float s = pow2_to(am, 14);
            fac[e] = p.scale_log2 / s;
            uint32_t d[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) q_to_f16(u[i], s, d + 4 * i);
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // MMA i sums over bytes 4i..4i+3 of the lane's 32
                qa[i][e] = d[2 * i];
                qa[i][2 + e] = d[2 * i + 1];
            }
        }
        float o[16][4];
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, sref = 0.0f;
        // scales of a step's two 16-key halves, read a step ahead
        const float* ks = p.k_scale + it.b * p.s_seq + hk;
        const float* vs = p.v_scale + it.b * p.s_seq + hk;
        const int last = (it.nkeys - 1) >> p.blk_shift;
        float kc[2], vc[2];
        auto scales = [&](int step) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int64_t at = min((step * kStep + 16 * e) >> p.blk_shift, last) * p.s_blk;
                kc[e] = __ldg(ks + at);
                vc[e] = __ldg(vs + at);
            }
        };
        scales(it.t0);
        for (int step = it.t0; step < it.t1; ++step) {
            const int st = used % kStages;
            const unsigned char* sk = ring + st * kStageBytes;
            const unsigned char* sv = sk + kTile;
            const int key0 = step * kStep;
            const float k0 = kc[0], k1 = kc[1], v0 = vc[0], v1 = vc[1];
            if (step + 1 < it.t1) scales(step + 1);
            if (ok && !__all_sync(0xffffffffu, mbar_wait_sleep(&bar[warp][st], (used / kStages) & 1))) {
                // a copy that never landed: no more reading, nothing is refilled,
                // and the other copies land before shared memory goes away
                ok = false;
                if (lane == 0) raise_status(p.status, kDevTimeout);
                for (int f = used + 1; f < filled; ++f) mbar_wait_sleep(&bar[warp][f % kStages], (f / kStages) & 1);
            }
            ++used;
            if (!ok) continue;
            // ---- scores: rows g, g + 8; keys 8 nt + 2t, + 1 ----
            float s[4][4];
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
                const unsigned char* row = sk + (nt * 8 + g) * kKvqHeadDim;
                const uint4 a = *reinterpret_cast<const uint4*>(row + ((t ^ g) << 4));
                const uint4 b = *reinterpret_cast<const uint4*>(row + (((t + 4) ^ g) << 4));
                const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    mma_f16(s[nt], qa[i], e4m3_to_f16x2(w[i] & 0xffffu), e4m3_to_f16x2(w[i] >> 16));
            }
            const bool edge = key0 + kStep > it.L;
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                const float kk = nt < 2 ? k0 : k1;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x = s[nt][e] * (kk * fac[e >> 1]);
                    if (edge) {
                        const int j = key0 + nt * 8 + 2 * t + (e & 1) - it.L;  // tree slot (< 0: prefix)
                        if (j >= 0 && !(j < 32 && ((see[e >> 1] >> j) & 1u))) x = -INFINITY;
                    }
                    s[nt][e] = x;
                    mx[e >> 1] = fmaxf(mx[e >> 1], x);
                }
            }
            // ---- running maximum and reference V scale, raised only by more than 2^8 (2^4): weights stay below 2^12 ----
            float al[2] = {1.0f, 1.0f};
            bool raise = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
                mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
                if (mx[e] > m[e] + 8.0f || (m[e] == -INFINITY && mx[e] > -INFINITY)) {
                    al[e] = m[e] == -INFINITY ? 0.0f : ex2_approx(m[e] - mx[e]);
                    m[e] = mx[e];
                    l[e] *= al[e];
                    raise = true;
                }
            }
            const float vm = fmaxf(v0, v1);
            if (vm > 16.0f * sref) {  // uniform over the warp
                const float r = sref / vm;
                al[0] *= r;
                al[1] *= r;
                sref = vm;
                raise = true;
            }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    o[j][0] *= al[0];
                    o[j][1] *= al[0];
                    o[j][2] *= al[1];
                    o[j][3] *= al[1];
                }
            }
            const float rv[2] = {v0 / sref, v1 / sref};
            const float mu[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
            uint32_t pa[2][4];  // weights as A fragments, 16 keys each
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] = ex2_approx(s[nt][e] - mu[e >> 1]);
                    l[e >> 1] += w[e];
                    w[e] *= rv[nt >> 1];
                }
                pa[nt >> 1][(nt & 1) * 2] = pack_f16(w[0], w[1]);
                pa[nt >> 1][(nt & 1) * 2 + 1] = pack_f16(w[2], w[3]);
            }
            // ---- O += P V: keys 16 hf + {2t, 2t+1, 8+2t, 8+2t+1}, columns 16 g .. 16 g + 15 ----
            const bool tail = key0 + kStep > it.nkeys;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                uint4 u[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = hf * 16 + (e >> 1) * 8 + 2 * t + (e & 1);
                    u[e] = *reinterpret_cast<const uint4*>(sv + key * kKvqHeadDim + ((g ^ (key & 7)) << 4));
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
                    mma_f16(o[4 * i], pa[hf], e4m3_to_f16x2(a & 0xffffu), e4m3_to_f16x2(b & 0xffffu));
                    mma_f16(o[4 * i + 1], pa[hf], e4m3_to_f16x2(a >> 16), e4m3_to_f16x2(b >> 16));
                    mma_f16(o[4 * i + 2], pa[hf], e4m3_to_f16x2(c & 0xffffu), e4m3_to_f16x2(d & 0xffffu));
                    mma_f16(o[4 * i + 3], pa[hf], e4m3_to_f16x2(c >> 16), e4m3_to_f16x2(d >> 16));
                }
            }
            __syncwarp();  // every lane has read the stage
            fill();
        }
        // ---- the piece's rows: columns 32t .. 32t+31 of rows g, g + 8 ----
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            const int r = g + 8 * e;
            if (r >= rows) continue;
            if (it.whole()) {
                const int slot = r / p.G;
                const bool live = ok && slot < it.n && l[e] > 0.0f;
                const float inv = live ? sref / l[e] : 0.0f;
                uint4* dst = reinterpret_cast<uint4*>(
                    p.out + ((static_cast<size_t>(it.b) * p.s.T + slot) * p.Hq + hk * p.G + (r - slot * p.G)) * kKvqHeadDim +
                    32 * t);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = (c & 1) * 8 + 2 * i;
                        w[i] = live ? pack_bf16(o[j][2 * e + (c >> 1)] * inv, o[j + 1][2 * e + (c >> 1)] * inv) : 0u;
                    }
                    dst[c] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            } else {
                const size_t row = static_cast<size_t>(it.slot(worker)) * p.part.rows + r;
                float4* dst = reinterpret_cast<float4*>(p.part.o + row * kKvqHeadDim + 32 * t);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const int j = (c & 3) * 4, x = 2 * e + (c >> 2);
                    dst[c] = make_float4(o[j][x] * sref, o[j + 1][x] * sref, o[j + 2][x] * sref, o[j + 3][x] * sref);
                }
                if (t == 0) {
                    p.part.ml[2 * row] = ok ? m[e] : -INFINITY;
                    p.part.ml[2 * row + 1] = ok ? l[e] : 0.0f;
                }
            }
        }
    }
}

// ------------------------------------------------------------------ merge ---

constexpr int kMergeWarps = 8;
constexpr int kMergeAlone = 4;  // most pieces that one warp combines by itself

// The cut item that worker w began: O = sum_i 2^(m_i - M) O_i over
// sum_i 2^(m_i - M) l_i of its pieces i (worker w's in slot 2w + 1, w + i's in
// slot 2 (w + i)).
struct CutItem {
    int np;  // pieces; 0: worker w began none that was cut
    int b, sub, n;
};

__device__ __forceinline__ CutItem cut_item(const KvqSched& s, int w) {  // whole warp
    CutItem c{0, 0, 0, 0};
    const long long total = kvq_total(s), chunk = kvq_chunk(s, total);
    const long long end = (w + 1) * chunk;
    if (w * chunk >= total || end >= total) return c;  // the last worker's items end with it
    long long base;
    const int b = kvq_find(s, end - 1, &base);
    const KvqSeq q = kvq_seq(s, b);
    const int sub = static_cast<int>((end - 1 - base) / q.len);
    const long long g0 = base + static_cast<long long>(sub) * q.len;
    const long long t1 = end - g0 - s.ov, t0 = w * chunk - g0 - s.ov;
    if (t1 <= 0 || t1 >= q.nt || t0 > 0) return c;  // not cut, or begun by an earlier worker
    c.np = static_cast<int>((g0 + s.ov + q.nt - 1) / chunk) - w + 1;
    c.b = b;
    c.sub = sub;
    c.n = q.n;
    return c;
}

// Running combination of a row's pieces, four columns per lane.
struct RowSum {
    float m = -INFINITY, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    __device__ __forceinline__ void add(float pm, float pl, const float4& x) {
        // a piece in which the row saw nothing: maximum -inf, O 0
        const float M = fmaxf(m, pm);
        const float a = m == -INFINITY ? 0.0f : ex2_approx(m - M), c = pm == -INFINITY ? 0.0f : ex2_approx(pm - M);
        m = M;
        l = l * a + pl * c;
        o = make_float4(o.x * a + x.x * c, o.y * a + x.y * c, o.z * a + x.z * c, o.w * a + x.w * c);
    }
};

__device__ __forceinline__ void merge_store(const KvqMergeParams& p, const CutItem& c, int r, const RowSum& s, int lane) {
    const int hk = c.sub / p.n_rb, row = (c.sub - hk * p.n_rb) * p.part.rows + r;
    const int slot = row / p.G;
    if (slot >= p.T) return;  // past the (sequence, KV head)'s rows
    const bool live = slot < c.n && s.l > 0.0f;
    const float inv = live ? 1.0f / s.l : 0.0f;
    uint2* dst = reinterpret_cast<uint2*>(
        p.out + ((static_cast<size_t>(c.b) * p.T + slot) * p.Hq + static_cast<size_t>(hk) * p.G + (row - slot * p.G)) * kKvqHeadDim);
    dst[lane] = live ? make_uint2(pack_bf16(s.o.x * inv, s.o.y * inv), pack_bf16(s.o.z * inv, s.o.w * inv))
                     : make_uint2(0u, 0u);
}

// A CTA serves the items that eight neighbouring workers began (decode: few
// rows) or one worker's (128 rows, blockIdx.y taking some of them). Which those are
// comes from the lengths alone and is found while the attention kernel still
// runs. With 128 rows a warp takes whole rows. Decode items of up to four pieces go
// to one warp each; those of many (few long sequences) are shared by all
// eight warps, row by row.
__global__ void __launch_bounds__(kMergeWarps * 32) kvq_merge_kernel(KvqMergeParams p, int per_cta, int rows_per_cta) {
    __shared__ CutItem items[kMergeWarps];
    __shared__ float4 so[kMergeWarps][32];
    __shared__ float2 sml[kMergeWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int w0 = blockIdx.x * per_cta;
    if (warp < per_cta) {
        const CutItem c = w0 + warp < p.s.workers ? cut_item(p.s, w0 + warp) : CutItem{0, 0, 0, 0};
        if (lane == 0) items[warp] = c;
    }
    __syncthreads();
    pdl_wait_prior();
    pdl_launch_dependents();
    const int r0 = blockIdx.y * rows_per_cta, r1 = min(p.part.rows, r0 + rows_per_cta);
    const float2* ml = reinterpret_cast<const float2*>(p.part.ml);
    const float4* po = reinterpret_cast<const float4*>(p.part.o);
    auto slot_row = [&](int w, int i, int r) {
        return static_cast<size_t>(i == 0 ? 2 * w + 1 : 2 * (w + i)) * p.part.rows + r;
    };
    const bool decode = per_cta > 1;
    for (int e = 0; e < per_cta; ++e) {
        const CutItem c = items[e];
        if (c.np == 0 || (decode && (c.np > kMergeAlone || e != warp))) continue;
        // decode: item e belongs to warp e; else its rows are dealt over the warps
        for (int r = decode ? r0 : r0 + warp; r < r1; r += decode ? 1 : kMergeWarps) {
            RowSum s;
            for (int i0 = 0; i0 < c.np; i0 += kMergeAlone) {
                float2 a[kMergeAlone];
                float4 x[kMergeAlone];
#pragma unroll
                for (int i = 0; i < kMergeAlone; ++i) {
                    if (i0 + i >= c.np) break;
                    const size_t at = slot_row(w0 + e, i0 + i, r);
                    a[i] = __ldcg(ml + at);
                    x[i] = __ldcg(po + at * 32 + lane);
                }
#pragma unroll
                for (int i = 0; i < kMergeAlone; ++i)
                    if (i0 + i < c.np) s.add(a[i].x, a[i].y, x[i]);
            }
            merge_store(p, c, r, s, lane);
        }
    }
    for (int e = 0; e < per_cta; ++e) {
        const CutItem c = items[e];
        if (!decode || c.np <= kMergeAlone) continue;  // uniform over the CTA
        for (int r = r0; r < r1; ++r) {
            RowSum s;
#pragma unroll 4
            for (int i = warp; i < c.np; i += kMergeWarps) {
                const size_t at = slot_row(w0 + e, i, r);
                const float2 a = __ldcg(ml + at);
                const float4 x = __ldcg(po + at * 32 + lane);
                s.add(a.x, a.y, x);
            }
            so[warp][lane] = s.o;
            if (lane == 0) sml[warp] = make_float2(s.m, s.l);
            __syncthreads();
            if (warp == 0) {
                for (int i = 1; i < kMergeWarps; ++i) s.add(sml[i].x, sml[i].y, so[i][lane]);
                merge_store(p, c, r, s, lane);
            }
            __syncthreads();
        }
    }
}

}  // namespace

cudaError_t launch_kvq_merge(const KvqMergeParams& p, cudaStream_t stream) {
    const bool decode = p.part.rows <= kKvqDecodeRows;
    const int per_cta = decode ? kMergeWarps : 1, rows_per_cta = decode ? p.part.rows : 32;
    return launch_pdl(kvq_merge_kernel,
                      dim3((p.s.workers + per_cta - 1) / per_cta, (p.part.rows + rows_per_cta - 1) / rows_per_cta),
                      dim3(kMergeWarps * 32), 0, stream, p, per_cta, rows_per_cta);
}

KvqSched kvq_decode_sched(int B, int T, int max_len, int Hkv) {
    return KvqSched{nullptr, nullptr, B, T, max_len, Hkv, kStep, 2, kKvqSms * kWarps, 4};
}

cudaError_t launch_kvq_decode(const KvqDims& kv, const KvqAttnParams& p, const void* kbase, const void* vbase,
                              cudaStream_t stream) {
    CUtensorMap tk, tv;
    if (!make_map_codes(&tk, kbase, kv, kStep) || !make_map_codes(&tv, vbase, kv, kStep)) return cudaErrorInvalidValue;
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kvq_decode_kernel), kSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kvq_decode_kernel, dim3(kKvqSms), dim3(kWarps * 32), kSmem, stream, tk, tv, p);
}

}  // namespace eagle
