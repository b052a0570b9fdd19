// LM head with 4-bit weights and group scales (sm_103a): logits [M, V] =
// hidden [M, H] (bf16) x weight [V, H]^T, weight[v, h] = (c - 8) * scale of
// (v, h / group). ["EAGLE" notes, EAGLE 方法: the draft model reuses the target
// model's LM head]; the 4-bit form is not on the pages.
//
// With the few rows of a small batch the weight's bytes are the cost (V*H/2,
// a quarter of the 16-bit head's), 4 M flops a byte. Per byte there is little
// time: two products per code and row, so the codes are taken from registers:
//   - mma.sync m16n8k16 in fp16 with the weight as A (16 vocabulary rows) and
//     the hidden rows as B (8 per MMA). tcgen05 would need the weight in shared
//     or tensor memory: a code as a byte at least, twice its size, written and
//     read again on chip. (The e4m3 form of this instruction is no shortcut: it
//     runs as two fp16 ones behind conversions of both operands, 188 us at 8B.)
//   - the fp16 number with the bits 0000 0000 0000 cccc is c 2^-24, and with
//     the code four bits higher 16 times that (subnormals, which the tensor core
//     takes exactly), so a word's eight codes become four operand registers in five
//     instructions: w & 0x000f000f and w & 0x00f000f0, the same of w >> 8. (To bf16
//     numbers c - 8 it takes eleven: 112 us at 8B.) The hidden entries of the higher
//     codes are 16 times smaller, and the 8 that a code is above its weight is
//     taken off by the accumulator's start: -8 times the group's sum of the hidden row.
//   - a hidden row is scaled by the power of two that brings its largest element
//     into [2^14, 2^15): its bf16 entries are fp16 numbers then, exact down to
//     2^-28 of the largest.
//   - a group's sum is multiplied by its scale in fp32: no rounding of a weight.
//   - the hidden dimension is summed over in an order in which a lane holds
//     32 neighbouring entries of a weight row (one 16-byte load of codes per
//     128 entries) and the hidden rows are laid out in shared memory in that
//     order once per CTA.
// One persistent CTA per SM takes an equal, contiguous range of the
// vocabulary in tiles of 64 or 32 rows; its eight MMA warps split the hidden
// dimension (warp w: the 128-wide slices w, w + 8, ...), so that each works
// alone, streaming its slices of one tile after the other through its own
// ring of TMA tiles (filled by a warp for all eight rings: a copy's issue takes
// 400 cycles) and reading a slice's codes while the one before is multiplied;
// three more warps add the eight partial sums of a finished tile and write the
// logits while the next tile streams.
//
// Measured: 8 rows, H = 8192, V = 128256 (525 MB of codes): 108 us, 4.9 TB/s;
// 10 rows, H = 4096 (263 MB): 75.5 us, 3.5 TB/s. Bound by latency with two MMA
// warps per scheduler (their 168 registers allow no third beside the others):
// ten rows are two n-tiles of which the tensor pipe alone takes 28 us (8 cycles
// an MMA). Sixteen MMA warps of 96 registers: 119 and 128 us. More stages: no change.

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "attn_common.cuh"
#include "eagle_internal.cuh"
#include "quant_ptx.cuh"
#include "quant_ws.h"
#include "tc_ptx.cuh"

namespace eagle {
namespace {

constexpr int kMmaWarps = 8;
constexpr int kAddWarps = 3;
constexpr int kThreads = (kMmaWarps + kAddWarps + 1) * 32;  // and the copying warp: three warps per scheduler, 168 registers
constexpr int kSlice = 128;                // hidden entries of a slice
constexpr int kSliceBytes = kSlice / 2;    // codes of one row's slice
constexpr int kMaxStages = 4;
constexpr int kSms = 152;
constexpr int kMaxSmem = 227 * 1024 - 1024;  // dynamic, beside the barriers

struct QuantParams {
    int M, V, H, n_slice;
    int rows;        // hidden rows of a pass (blockIdx.y takes rows [y * rows, ...))
    int stages, bufs;  // ring stages of an MMA warp; buffers of partial sums
    int hid_stride;  // bytes of a hidden row in shared memory
    int c_stride;    // floats of a group's corrections
    const __nv_bfloat16* hidden;
    const __nv_bfloat16* scales;
    void* out;
    int* status;
};

// d = A B + (c0, c1, c0, c1): the first MMA of a group; then d += A B.
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1, float c0, float c1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %10, %11};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mma_next(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// A warp's bounded wait.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// Where the eight entries from `e` (within a slice, a multiple of 8) stand: lane
// t of a quad takes eight entries in each of the steps q = 0..3, neighbouring words
// of its codes for a group that spans the slice, quarters of the slice for the
// smaller groups. Piece (q, t), 16 bytes, is the (4 q + t)-th.
template <int GROUP>
__device__ __forceinline__ int piece_of(int e) {
    const int t = GROUP == 128 ? e >> 5 : GROUP == 64 ? (e >> 4) & 3 : (e >> 3) & 3;
    const int q = GROUP == 128 ? (e >> 3) & 3 : GROUP == 64 ? (e >> 6) * 2 + ((e >> 3) & 1) : e >> 5;
    return 4 * q + t;
}

// A row's NG scales of a slice as one load.
template <int NG>
struct ScaleWord {
    using type = unsigned short;
};
template <>
struct ScaleWord<2> {
    using type = uint32_t;
};
template <>
struct ScaleWord<4> {
    using type = uint2;
};
template <int NG>
__device__ __forceinline__ float scale_of(const typename ScaleWord<NG>::type& w, int i) {
    if constexpr (NG == 1) return __uint_as_float(static_cast<uint32_t>(w) << 16);
    else if constexpr (NG == 2) return __uint_as_float(i ? (w & 0xffff0000u) : (w << 16));
    else {
        const uint32_t x = i < 2 ? w.x : w.y;
        return __uint_as_float((i & 1) ? (x & 0xffff0000u) : (x << 16));
    }
}

// RT: vocabulary rows of a tile; NT: n-tiles of eight hidden rows.
template <int RT, int NT, int GROUP, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    lmhead_quant_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ CUtensorMap tm16, QuantParams p) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    __shared__ uint64_t bar_full[kMmaWarps][kMaxStages], bar_empty[kMmaWarps][kMaxStages], bar_red_full[2], bar_red_empty[2];
    constexpr int MT = RT / 16;
    constexpr int kStage = RT * kSliceBytes;
    constexpr int NG = kSlice / GROUP;  // groups of a slice
    using Scales = typename ScaleWord<NG>::type;
    constexpr int CS = RT + 4;          // a column of partial sums, padded: no bank conflicts
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int m0 = blockIdx.y * p.rows;
    const int rows = min(p.rows, p.M - m0);
    // rings of the MMA warps; hidden rows; corrections [group][c_stride]; the rows' factors;
    // partial sums of a tile, [buffer][warp][hidden row][CS]
    unsigned char* ring = smem + warp * p.stages * kStage;
    unsigned char* hid = smem + kMmaWarps * p.stages * kStage;
    float* corr = reinterpret_cast<float*>(hid + p.rows * p.hid_stride);
    float* fac = corr + p.n_slice * NG * p.c_stride;
    float* red = fac + 16;
    // this CTA's vocabulary rows, in units of 16
    const int units = (p.V + 15) / 16;
    const int u0 = static_cast<int>(static_cast<long>(units) * blockIdx.x / gridDim.x);
    const int u1 = static_cast<int>(static_cast<long>(units) * (blockIdx.x + 1) / gridDim.x);
    const int v0 = u0 * 16, v1 = u1 * 16;
    const int n_tiles = (v1 - v0 + RT - 1) / RT;
    if (threadIdx.x == 0) {
        for (int w = 0; w < kMmaWarps; ++w)
            for (int s = 0; s < p.stages; ++s) {
                mbar_init(&bar_full[w][s], 1);
                mbar_init(&bar_empty[w][s], 1);
            }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar_red_full[s], kMmaWarps);
            mbar_init(&bar_red_empty[s], kAddWarps);
        }
        fence_mbar_init();
    }
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait_prior();
    // The copying warp: lane w fills the ring of MMA warp w.
    const bool copies = warp == kMmaWarps + kAddWarps;
    const int total = copies && lane < kMmaWarps ? (p.n_slice - lane + kMmaWarps - 1) / kMmaWarps * n_tiles : 0;
    int filled = 0, f_tile = 0, f_slice = lane, f_stage = 0;
    uint32_t f_phase = 1;  // of the stage's release; the first round waits for nothing
    auto fill = [&]() {
        uint64_t* bar = &bar_full[lane][f_stage];
        unsigned char* dst = smem + (lane * p.stages + f_stage) * kStage;
        const int v = v0 + f_tile * RT;
        const int mts = min(MT, (v1 - v) / 16);  // a last tile of fewer rows: 16 at a time
        mbar_arrive_expect_tx(bar, mts * 16 * kSliceBytes);
        if (mts == MT)
            tma_load_2d(dst, &tm, f_slice * kSliceBytes, v, bar);
        else
            for (int i = 0; i < mts; ++i) tma_load_2d(dst + i * 16 * kSliceBytes, &tm16, f_slice * kSliceBytes, v + 16 * i, bar);
        ++filled;
        if (++f_stage == p.stages) {
            f_stage = 0;
            f_phase ^= 1;
        }
        f_slice += kMmaWarps;
        if (f_slice >= p.n_slice) {
            f_slice = lane;
            ++f_tile;
        }
    };
    // hidden rows into shared memory, a warp per row: its largest element, then pieces of eight
    // entries as fp16 in MMA order (0 4, 1 5, 2 6, 3 7), and the groups' corrections
    for (int m = warp; m < p.c_stride; m += kThreads / 32) {
        if (m >= rows) {  // columns of the last n-tile without a row
            for (int i = lane; i < p.n_slice * NG; i += 32) corr[i * p.c_stride + m] = 0.0f;
            continue;
        }
        const uint4* src = reinterpret_cast<const uint4*>(p.hidden + static_cast<size_t>(m0 + m) * p.H);
        const int pieces = p.H / 8;  // a multiple of 16: a group's lanes are in range together
        constexpr int kPer = kLmQuantMaxHidden / 8 / 32;
        uint4 u[kPer];
        uint32_t mx = 0u;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            if (32 * k >= pieces) break;
            u[k] = 32 * k + lane < pieces ? ld_prior(src + 32 * k + lane) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            if (32 * k >= pieces) break;
            mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(u[k].x & 0x7fff7fffu, u[k].y & 0x7fff7fffu),
                                       __vmaxu2(u[k].z & 0x7fff7fffu, u[k].w & 0x7fff7fffu)));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        mx = max(mx & 0xffffu, mx >> 16);
        const float scale = pow2_to(__uint_as_float(mx << 16), 14);
        // an infinity or NaN in the row makes its logits NaN
        if (lane == 0) fac[m] = mx < 0x7f80u ? 1.0f / scale : __uint_as_float(0x7fffffffu);
        unsigned char* row = hid + m * p.hid_stride;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            if (32 * k >= pieces) break;
            const int i = 32 * k + lane;
            const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = __uint_as_float((e & 1) ? (w[e >> 1] & 0xffff0000u) : (w[e >> 1] << 16)) * scale;
            float sum = ((x[0] + x[4]) + (x[1] + x[5])) + ((x[2] + x[6]) + (x[3] + x[7]));
            uint32_t h[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float f = (c & 1) ? 0x1p-4f : 1.0f;
                const __half2 y = __floats2half2_rn(x[c] * f, x[c + 4] * f);
                h[c] = *reinterpret_cast<const uint32_t*>(&y);
            }
#pragma unroll
            for (int o = 1; o < GROUP / 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (i >= pieces) continue;
            *reinterpret_cast<uint4*>(row + ((i >> 4) * 16 + piece_of<GROUP>((i & 15) * 8)) * 16) = make_uint4(h[0], h[1], h[2], h[3]);
            if (i % (GROUP / 8) == 0) corr[i / (GROUP / 8) * p.c_stride + m] = sum * -0x1p-21f;
        }
    }
    // the first copies behind the hidden rows: before them the rows' loads waited in their queue (1.5 us at 8B)
    if (copies)
        while (filled < min(p.stages, total)) fill();
    __syncwarp();
    __syncthreads();

    if (warp < kMmaWarps) {
        bool ok = true;
        // the lane's hidden row of each n-tile (columns without a row repeat the last one: nobody reads their sums)
        uint32_t h_at[NT];
#pragma unroll
        for (int b = 0; b < NT; ++b) h_at[b] = smem_u32(hid) + min(b * 8 + g, rows - 1) * p.hid_stride + t * 16;
        int st = 0;
        uint32_t phase = 0;
        // scales of rows g, g + 8 of every m-tile, a slice's NG together, read a slice ahead, also
        // over the border of a tile; rows past the vocabulary read its last one's
        Scales next[2 * MT];
        int r_tile = 0, r_slice = warp;
        auto read_scales = [&]() {
            if (r_tile >= n_tiles || warp >= p.n_slice) return;
            const int v = v0 + r_tile * RT, last = max(0, (p.V - 1 - v - g) >> 3);
            const __nv_bfloat16* src = p.scales + (static_cast<size_t>(v + g) * p.n_slice + r_slice) * NG;
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) next[i] = ld_prior(reinterpret_cast<const Scales*>(src + min(i, last) * 8 * p.n_slice * NG));
            r_slice += kMmaWarps;
            if (r_slice >= p.n_slice) {
                r_slice = warp;
                ++r_tile;
            }
        };
        read_scales();
        // codes of the warp's next slice, from its ring
        using Codes = uint32_t[MT][2][4];
        int left = warp < p.n_slice ? (p.n_slice - warp + kMmaWarps - 1) / kMmaWarps * n_tiles : 0;  // slices not read yet
        auto read_codes = [&](Codes& w) {
            if (left == 0 || !ok) return;
            --left;
            if (!warp_wait(&bar_full[warp][st], phase)) {
                ok = false;
                if (lane == 0) raise_status(p.status, kDevTimeout);
                return;
            }
            const uint32_t src = smem_u32(ring) + st * kStage;
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t row = src + (a * 16 + g + 8 * e) * kSliceBytes;
                    if (GROUP == 128) {
                        const uint4 x = lds128(row + t * 16);
                        w[a][e][0] = x.x, w[a][e][1] = x.y, w[a][e][2] = x.z, w[a][e][3] = x.w;
                    } else if (GROUP == 64) {
                        const uint2 x = lds64(row + t * 8), y = lds64(row + 32 + t * 8);
                        w[a][e][0] = x.x, w[a][e][1] = x.y, w[a][e][2] = y.x, w[a][e][3] = y.y;
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q) w[a][e][q] = lds32(row + q * 16 + t * 4);
                    }
                }
            __syncwarp();  // every lane has read the stage
            if (lane == 0) mbar_arrive(&bar_empty[warp][st]);
            if (++st == p.stages) {
                st = 0;
                phase ^= 1;
            }
        };
        float sum[MT][NT][4];
        auto clear = [&]() {
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int b = 0; b < NT; ++b) sum[a][b][0] = sum[a][b][1] = sum[a][b][2] = sum[a][b][3] = 0.0f;
        };
        // a tile's partial sums to the adding warps
        auto hand_over = [&](int tile) {
            const int buf = tile % p.bufs, turn = tile / p.bufs;
            if (ok && turn > 0 && !warp_wait(&bar_red_empty[buf], (turn - 1) & 1)) {
                ok = false;
                if (lane == 0) raise_status(p.status, kDevTimeout);
            }
            float* dst = red + (buf * kMmaWarps + warp) * p.rows * CS + g;
            if (ok) {
#pragma unroll
                for (int b = 0; b < NT; ++b)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int m = b * 8 + 2 * t + x;
                        if (m >= rows) continue;
#pragma unroll
                        for (int a = 0; a < MT; ++a)
#pragma unroll
                            for (int e = 0; e < 2; ++e) dst[m * CS + a * 16 + 8 * e] = sum[a][b][2 * e + x];
                    }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_red_full[buf]);
        };
        // a slice's products with the codes w; the next slice's go into `ahead` meanwhile
        auto slice_of = [&](int slice, const Codes& w, Codes& ahead) {
            Scales sc[2 * MT];
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) sc[i] = next[i];
            float acc[MT][NT][4];
            float2 c[NT];
            uint4 hb[2][NT];  // of step q and the next
            auto read_hidden = [&](int q) {
#pragma unroll
                for (int b = 0; b < NT; ++b) hb[q & 1][b] = lds128(h_at[b] + (slice * 16 + q * 4) * 16);
            };
            read_hidden(0);
            read_scales();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const bool first = q % (4 / NG) == 0;  // of a group
                if (first) {
#pragma unroll
                    for (int b = 0; b < NT; ++b) {
                        const uint2 x = lds64(smem_u32(corr) + ((slice * NG + q / (4 / NG)) * p.c_stride + b * 8 + 2 * t) * 4);
                        c[b] = make_float2(__uint_as_float(x.x), __uint_as_float(x.y));
                    }
                }
                if (q < 3) read_hidden(q + 1);
                if (q == 2) read_codes(ahead);
#pragma unroll
                for (int a = 0; a < MT; ++a) {
                    const uint32_t x = w[a][0][q], y = w[a][1][q], x8 = x >> 8, y8 = y >> 8;
                    constexpr uint32_t k0 = 0x000f000fu, k4 = 0x00f000f0u;
#pragma unroll
                    for (int b = 0; b < NT; ++b) {
                        const uint4& h = hb[q & 1][b];
                        if (first) mma_first(acc[a][b], x & k0, y & k0, x & k4, y & k4, h.x, h.y, c[b].x, c[b].y);
                        else mma_next(acc[a][b], x & k0, y & k0, x & k4, y & k4, h.x, h.y);
                    }
#pragma unroll
                    for (int b = 0; b < NT; ++b)
                        mma_next(acc[a][b], x8 & k0, y8 & k0, x8 & k4, y8 & k4, hb[q & 1][b].z, hb[q & 1][b].w);
                }
                if (q % (4 / NG) == 4 / NG - 1) {
                    const int gi = q / (4 / NG);
#pragma unroll
                    for (int a = 0; a < MT; ++a)
#pragma unroll
                        for (int b = 0; b < NT; ++b)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                sum[a][b][e] = fmaf(acc[a][b][e], scale_of<NG>(sc[2 * a + (e >> 1)], gi), sum[a][b][e]);
                }
            }
        };
        clear();
        if (left == 0) {  // fewer slices than warps: nothing to add
            for (int tile = 0; tile < n_tiles; ++tile) hand_over(tile);
        } else {
            Codes w0, w1;
            read_codes(w0);
            int tile = 0, slice = warp;
            auto step = [&](const Codes& w, Codes& ahead) {
                slice_of(slice, w, ahead);
                slice += kMmaWarps;
                if (slice < p.n_slice) return;
                hand_over(tile);
                clear();
                slice = warp;
                ++tile;
            };
            while (tile < n_tiles) {
                step(w0, w1);
                if (tile < n_tiles) step(w1, w0);
            }
        }
    } else if (!copies) {
        const int at = threadIdx.x - kMmaWarps * 32;
        for (int tile = 0; tile < n_tiles; ++tile) {
            const int buf = tile % p.bufs, turn = tile / p.bufs;
            const int v = v0 + tile * RT;
            const int nv = min(RT, min(v1, p.V) - v);  // rows of the tile inside the vocabulary (a multiple of 8)
            if (!warp_wait(&bar_red_full[buf], turn & 1)) {
                if (lane == 0) raise_status(p.status, kDevTimeout);
                break;
            }
            const float* src = red + buf * kMmaWarps * p.rows * CS;
            for (int i = at; i < rows * (RT / 2); i += kAddWarps * 32) {  // two vocabulary rows each
                const int m = i / (RT / 2), r = (i - m * (RT / 2)) * 2;
                if (r >= nv) continue;
                float x = 0.0f, y = 0.0f;
#pragma unroll
                for (int w = 0; w < kMmaWarps; ++w) {
                    const float2 s = *reinterpret_cast<const float2*>(src + (w * p.rows + m) * CS + r);
                    x += s.x;
                    y += s.y;
                }
                // 2^24 / scale in two powers of two, of which neither leaves fp32's range before the logit does
                const float f = fac[m], f0 = f < 1.0f ? f * 0x1p24f : 0x1p24f, f1 = f < 1.0f ? 1.0f : f;
                x = x * f0 * f1;
                y = y * f0 * f1;
                const size_t o = static_cast<size_t>(m0 + m) * p.V + v + r;
                if (BF16) *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + o) = pack_bf16(x, y);
                else *reinterpret_cast<float2*>(static_cast<float*>(p.out) + o) = make_float2(x, y);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_red_empty[buf]);
        }
    } else {
        uint32_t polls = 0;
        bool ok = true;
        while (__any_sync(0xffffffffu, ok && filled < total)) {
            bool did = false;
            if (ok && filled < total) {
                if (mbar_test_wait(&bar_empty[lane][f_stage], f_phase)) {
                    fill();
                    did = true;
                    polls = 0;
                } else if (++polls > (1u << 21)) {  // that MMA warp gave up: its copies land before shared memory goes away
                    ok = false;
                    for (int f = max(0, filled - p.stages); f < filled; ++f)
                        mbar_wait(&bar_full[lane][f % p.stages], (f / p.stages) & 1, 1u << 16);
                }
            }
            if (!__any_sync(0xffffffffu, did)) __nanosleep(32);
        }
    }
}

// A 2-D map of the codes: (bytes of a row, row), boxes of one slice x `rows` rows.
bool make_map(CUtensorMap* m, const void* codes, int V, int H, int rows) {
    auto fn = tensor_map_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(H / 2), static_cast<cuuint64_t>(V)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(H / 2)};
    const cuuint32_t box[2] = {kSliceBytes, static_cast<cuuint32_t>(rows)};
    const cuuint32_t estride[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box, estride,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Shared memory of a pass of `rows` hidden rows with RT-row tiles, `stages` per ring and `bufs` buffers of partial sums.
int smem_bytes(int rows, int H, int group, int RT, int stages, int bufs) {
    return kMmaWarps * stages * RT * kSliceBytes + rows * (2 * H + 64) + ((H / group) * ((rows + 7) & ~7) + 16) * 4 +
           bufs * kMmaWarps * rows * (RT + 4) * 4 + 128;
}

template <int RT, int NT, int GROUP, bool BF16>
cudaError_t launch(const QuantParams& p, const void* codes, int smem, cudaStream_t stream) {
    CUtensorMap tm, tm16;
    if (!make_map(&tm, codes, p.V, p.H, RT) || !make_map(&tm16, codes, p.V, p.H, 16)) return cudaErrorInvalidValue;
    auto kernel = lmhead_quant_kernel<RT, NT, GROUP, BF16>;
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), smem);
    if (e != cudaSuccess) return e;
    const int units = (p.V + 15) / 16;
    return launch_pdl(kernel, dim3(std::min(kSms, units), (p.M + p.rows - 1) / p.rows), dim3(kThreads),
                      static_cast<size_t>(smem), stream, tm, tm16, p);
}

template <int RT, int NT>
cudaError_t launch_group(const QuantParams& p, int group, bool bf16, const void* codes, int smem, cudaStream_t s) {
    if (group == 128) return bf16 ? launch<RT, NT, 128, true>(p, codes, smem, s) : launch<RT, NT, 128, false>(p, codes, smem, s);
    if (group == 64) return bf16 ? launch<RT, NT, 64, true>(p, codes, smem, s) : launch<RT, NT, 64, false>(p, codes, smem, s);
    return bf16 ? launch<RT, NT, 32, true>(p, codes, smem, s) : launch<RT, NT, 32, false>(p, codes, smem, s);
}

// ------------------------------------------------------------------- pack ---

// One lane per eight entries; group / 8 neighbouring lanes share a scale. Run once
// per model and not made fast: 637 us at V = 128256, H = 4096 (1.3 GB moved, 198 us
// at the copy's rate).
__global__ void __launch_bounds__(256) lmhead_quant_pack_kernel(long pieces, int group, const uint4* weight,
                                                                uint32_t* __restrict__ codes,
                                                                __nv_bfloat16* __restrict__ scales) {
    pdl_launch_dependents();
    pdl_wait_prior();
    const int lanes = group / 8;
    // pieces is a multiple of lanes (<= 16), so a group's lanes are in range together
    for (long i = static_cast<long>(blockIdx.x) * 256 + threadIdx.x; i - (threadIdx.x & 31) < pieces; i += 256l * gridDim.x) {
        const bool in = i < pieces;
        const uint4 u = in ? weight[i] : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        float x[8], am = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = __uint_as_float((e & 1) ? (w[e >> 1] & 0xffff0000u) : (w[e >> 1] << 16));
            am = fmaxf(am, fabsf(x[e]));
        }
        for (int o = 1; o < lanes; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
        const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(am, 7.0f));
        const float s = __bfloat162float(sb);
        uint32_t c = 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float q = s > 0.0f ? rintf(__fdiv_rn(x[e], s)) : 0.0f;
            c |= (static_cast<uint32_t>(8 + static_cast<int>(fminf(fmaxf(q, -7.0f), 7.0f))) & 15u) << (4 * e);
        }
        if (in) {
            codes[i] = c;
            if (i % lanes == 0) scales[i / lanes] = sb;
        }
    }
}

}  // namespace

cudaError_t launch_lmhead_quant(int M, int V, int H, int group, const void* hidden, const void* codes,
                                const void* scales, int out_dtype, void* out, int* status, cudaStream_t stream) {
    QuantParams p{};
    p.M = M;
    p.V = V;
    p.H = H;
    p.n_slice = H / kSlice;
    p.hid_stride = 2 * H + 64;  // rows 64 bytes apart modulo 128: no bank conflicts between neighbouring rows
    p.hidden = static_cast<const __nv_bfloat16*>(hidden);
    p.scales = static_cast<const __nv_bfloat16*>(scales);
    p.out = out;
    p.status = status;
    // Up to 16 hidden rows per pass, 8 when 16 (or all, if fewer) do not fit beside two stages
    // of the rings. Tiles of 64 vocabulary rows (a load of a hidden piece serves four MMAs), 32
    // when 64 do not fit, or with two n-tiles, whose sums leave no registers for the next slice's
    // codes of 64 rows (103 against 77 us at 8B); a second buffer of partial sums and more stages
    // where there is room.
    const bool bf16 = out_dtype == 1;
    auto run = [&](int rows, int RT, auto fn, cudaError_t* e) -> bool {
        int st = 2, nb = 1;
        if (smem_bytes(rows, H, group, RT, st, nb) > kMaxSmem) return false;
        if (smem_bytes(rows, H, group, RT, st, 2) <= kMaxSmem) nb = 2;
        while (st < kMaxStages && smem_bytes(rows, H, group, RT, st + 1, nb) <= kMaxSmem) ++st;
        p.rows = rows;
        p.c_stride = (rows + 7) & ~7;
        p.stages = st;
        p.bufs = nb;
        *e = fn(p, group, bf16, codes, smem_bytes(rows, H, group, RT, st, nb), stream);
        return true;
    };
    cudaError_t e = cudaErrorInvalidValue;
    if (M > 8) {
        const int rows = std::min(M, 16);
        if (run(rows, 32, launch_group<32, 2>, &e)) return e;
    }
    const int rows = std::min(M, 8);
    if (run(rows, 64, launch_group<64, 1>, &e) || run(rows, 32, launch_group<32, 1>, &e)) return e;
    return e;
}

cudaError_t launch_lmhead_quant_pack(int V, int H, int group, const void* weight, void* codes, void* scales,
                                     cudaStream_t stream) {
    const long pieces = static_cast<long>(V) * H / 8;
    const unsigned grid = static_cast<unsigned>(std::min<long>((pieces + 255) / 256, 152 * 16));
    return launch_pdl(lmhead_quant_pack_kernel, dim3(grid), dim3(256), 0, stream, pieces, group,
                      static_cast<const uint4*>(weight), static_cast<uint32_t*>(codes),
                      static_cast<__nv_bfloat16*>(scales));
}

}  // namespace eagle
