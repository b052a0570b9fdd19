// Product of rows and weights of 8-bit codes with power-of-two scales
// (sm_103a): eagle_linear_fp8, out[m, n] = sum_k x[m, k] w[n, k].
//
// The tensor cores take the scales themselves (tcgen05.mma kind::mxf8f6f4 with
// block scaling): each MMA of K = 32 multiplies its e4m3 products by the two
// operands' scale bytes (E8M0) and adds them to fp32 sums in tensor memory, so
// no partial sum is read back to be scaled. A scale covers 128 entries of K,
// four MMAs that name the same byte of a scale word; a word holds the bytes of
// four blocks, K = 512.
//
// As in the 16-bit LM head the product is computed as w x^T: 128 weight rows
// fill the MMA's 128 lanes, Nr rows of x its columns, so few rows cost few
// columns.
//   tile            weight rows 128 vt .. against a chunk of x rows, summed over
//                   K in stages of 128 codes (128-byte rows, 128B swizzle)
//   warp 0          streams the boxes of w and x into a ring (TMA)
//   warp 1          issues the MMAs into fp32 accumulators in tensor memory and
//                   the copies of the scale words into it (tcgen05.cp)
//   warp 2          lays the scale words out for those copies, one group of
//                   K = 512 after the other
//   warps 4..11     read the accumulators and store the outputs
// Rows and columns past the operands' ends arrive as zeros and are not stored.
//
// Many rows (CG = 2): two CTAs share an MMA of 256 weight rows (cta_group::2),
// each holding its 128 of them and half of the rows of x; the first of the pair
// issues. A stage's weights meet two accumulators of Nr <= 224 rows each, so a
// tile is 256 x 448.
// Few rows (CG = 1, up to 224): one accumulator per tile, two tiles deep; the CTAs
// share the weight's rows evenly. Where there are at most half as many tiles as
// SMs a cluster's CTAs each take a part of a tile's K and their sums meet in
// distributed shared memory, added in the CTAs' order.
//
// What bounds it. Few rows: HBM and some 4 us that a launch costs (10 rows
// against 128256 x 4096: 82 to 84 us, 93 to 95% of HBM; 64 rows against 4096 x 4096
// 7.9 us). Many: the weight comes from L2 once
// for each row chunk of a tile, and L2 gives 7.2 TB/s of lines that no two SMs ask
// for together, hence the two accumulators (with one, 225 us for the next case);
// then the card's power: 640 rows against 128256 x 4096 205 to 213 us at the start
// of a series (3.2 PFLOP/s at 1.7 GHz), 239 to 246 in a long one (1.5 GHz), 177 us on
// zeros (1.95 GHz; 164 us without loads and stores); 4001 rows against 14336 x 4096
// 131 to 134 us, 151 to 154 in a long series, 117 on zeros (4.0 PFLOP/s). Copies of
// x's boxes shared by a cluster of two pairs were slower: 144 SMs, and four CTAs in
// step (263 us on zeros).

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "eagle_internal.cuh"
#include "eagle_ws.h"
#include "quant_ptx.cuh"
#include "quant_ws.h"
#include "tc_ptx.cuh"

namespace eagle {
namespace {

constexpr int kTileN = 128;   // weight rows of a CTA's tile (the MMA's M is 128 a CTA)
constexpr int kStageK = 128;  // codes of K of a stage
constexpr int kGroup = 4;     // stages of a word of scales, K = 512
constexpr int kMaxNr = 224;   // rows of x of an accumulator (MMA N): two accumulators and the scales fit in 512 columns
constexpr int kMaxNrFew = 128;  // (CG = 1, few tiles)
constexpr int kPartRows = 16; // (CG = 1) weight rows in which they are dealt to the CTAs
constexpr int kMaxStages = 8;
constexpr int kSfSlots = 3;   // groups of scale words on their way
constexpr int kSfBytes = 512; // scale words of 128 rows and K = 512
constexpr int kEpiWarps = 8;
constexpr int kLinThreads = 128 + 32 * kEpiWarps;
constexpr int kWBytes = kTileN * kStageK;
constexpr int kOutBytes = 32768;  // (CG = 2) outputs on their way to memory: four boxes (fp32: two) a warp
constexpr int kSmemBudget = 226 * 1024;
constexpr int kMaxSplit = 8;
constexpr int kMaxDevices = 64;
// An MMA cuts what it adds to a sum to fp32's last place, so long sums come out smaller (K = 8192: 1.3e-6 of the
// outputs' norm): fp32 outputs are summed in tensor memory over K = 2048 (CG = 1) or 4096, and those sums in fp32.
constexpr int kF32Chunk1 = 16, kF32Chunk2 = 32;

struct LinParams {
    int M, N, K;
    int Nr;           // rows of x of an accumulator
    int nrc;          // row chunks (of a tile's accumulators)
    int ntiles;
    int nwt;          // 128-row tiles of the weight
    int split;        // CTAs of a cluster that share a tile's K (CG = 1)
    int nk;           // stages of a tile
    int per;          // stages of a CTA (whole groups)
    int chunk;        // stages summed in tensor memory (whole groups)
    int stages;       // of the ring
    int stage_bytes;
    int sf_blocks;    // 128-row blocks of scale words of an accumulator's rows
    int sf_row_words; // scale words of a row
    uint32_t acc_stride, sf_col, sf_cols, tmem_cols;
    int bulk_out;     // the output's rows allow bulk stores (16-byte rows)
    const uint32_t *x_scales, *w_scales;
    void* out;
    int* status;
};

// Instruction descriptor of kind::mxf8f6f4: A and B e4m3 (0), both K-major, N >> 3 at bits 17-22,
// E8M0 scales (bit 23), M >> 4 at bits 24-28; the scale word's byte for B at bits 4-5, for A at 29-30.
__host__ __device__ constexpr uint32_t idesc_mxf8(int M, int N) {
    return (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(M >> 4) << 24);
}
// Operands by the low words of their descriptors (address and leading offset); the high word is the same for all.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
template <int CG>
__device__ __forceinline__ void mma_mxf8(uint32_t tmem_d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, int accum) {
    if (CG == 1)
        asm volatile(
            "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %6, 0;\n mov.b64 da, {%1, %7};\n mov.b64 db, {%2, %7};\n"
            " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], da, db, %3, [%4], [%5], p;\n}" ::"r"(tmem_d),
            "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accum), "r"(kDescHi)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %6, 0;\n mov.b64 da, {%1, %7};\n mov.b64 db, {%2, %7};\n"
            " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], da, db, %3, [%4], [%5], p;\n}" ::"r"(tmem_d),
            "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accum), "r"(kDescHi)
            : "memory");
}
// Descriptor of 32 rows of 16 bytes, one after the other (no swizzle): 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t sf_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 16) |
           (static_cast<uint64_t>(128 >> 4) << 32) | (1ull << 46);
}
// Those 512 bytes into four columns of tensor memory, the same in each quarter of its lanes (of a
// pair: each CTA's bytes into its own).
template <int CG>
__device__ __forceinline__ void copy_sf(uint32_t taddr, uint64_t desc) {
    if (CG == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// An arrival on `bar` (of a pair: on both CTAs' barriers) when the MMAs and copies so far have ended.
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
    if (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"(static_cast<uint16_t>(3))
            : "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
// On a barrier of the pair's first CTA, for what this thread has written to its own CTA's memory ...
__device__ __forceinline__ void arrive_at(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// ... and without anything written. (That release takes so long that scales came late with it: 10 rows against
// 128256 x 4096 92 us, 82 with arrivals within the CTA; 640 rows of zeros 193, 181.)
__device__ __forceinline__ void arrive_at_relaxed(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// A bounded wait by a whole warp, whose lanes leave it together. PEER: for what the other CTA of a pair wrote, too (the
// wider scope at every wait: 640 rows of zeros against 128256 x 4096 181 us, 177 without). Without the hint of how long
// to sleep: that cost some 30 clocks a stage.
template <bool PEER = false>
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) {
    for (uint32_t i = 0; i < (1u << 21); ++i) {
        uint32_t ok;
        if (PEER)
            asm volatile(
                "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
                " selp.u32 %0, 1, 0, p;\n}"
                : "=r"(ok)
                : "r"(bar), "r"(parity)
                : "memory");
        else
            asm volatile(
                "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
                : "=r"(ok)
                : "r"(bar), "r"(parity)
                : "memory");
        if (__all_sync(0xffffffffu, ok)) return true;
    }
    return false;
}
// The same for warps that wait long.
__device__ __forceinline__ bool wait_warp_sleep(uint32_t bar, uint32_t parity) {
    for (uint32_t i = 0; i < (1u << 16); ++i) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(20000u)
            : "memory");
        if (__all_sync(0xffffffffu, ok)) return true;
    }
    return false;
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}
template <int CG>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
    else  // into this CTA's memory, counted on the barrier of the pair's first
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
}
__device__ __forceinline__ void prefetch_box(const CUtensorMap* map, int c0, int c1) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(c0),
                 "r"(c1)
                 : "memory");
}
__device__ __forceinline__ void store_remote(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 16 rows of the output from `o` on, rows n elements apart, `live` of them.
template <typename T>
__device__ __forceinline__ void store_rows(T* o, int64_t n, int live, const float* x) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        if (j < live) {
            if (sizeof(T) == 2) *reinterpret_cast<__nv_bfloat16*>(o) = __float2bfloat16_rn(x[j]);
            else *reinterpret_cast<float*>(o) = x[j];
        }
        o += n;
    }
}
// A box of the output from shared memory, stored or (fp32) added to what is there.
__device__ __forceinline__ void store_block(const CUtensorMap* map, uint32_t src, int c0, int c1, bool add) {
    if (add)
        asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                         reinterpret_cast<uint64_t>(map)),
                     "r"(c0), "r"(c1), "r"(src)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                         reinterpret_cast<uint64_t>(map)),
                     "r"(c0), "r"(c1), "r"(src)
                     : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// Blocks of 16 columns of an accumulator that the warps of one half read.
constexpr int kHalfBlocks = kMaxNr / 32;
__device__ __forceinline__ int half_first(int Nr, int half) { return half ? (Nr / 16 + 1) / 2 : 0; }
__device__ __forceinline__ int half_count(int Nr, int half) { return half ? Nr / 32 : (Nr / 16 + 1) / 2; }

// CG: CTAs that share an MMA, and accumulators of a tile. tm_more: the output's map (CG = 2), or the weight's with
// boxes of kPartRows rows (CG = 1).
template <int CG, bool BF16>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_fp8_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                      const __grid_constant__ CUtensorMap tm_more, const LinParams p) {
    constexpr int NSUB = CG;  // accumulators of a tile
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ __align__(8) uint64_t bar_full[kMaxStages], bar_empty[kMaxStages], bar_sf_full[kSfSlots],
        bar_sf_empty[kSfSlots], bar_acc_full[2], bar_acc_empty[2];
    __shared__ uint32_t tmem_holder;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ncta = CG == 2 ? 2 : p.split;  // CTAs of the cluster
    const int rank = blockIdx.x % ncta;
    const int lead = CG == 2 ? 0 : rank;     // who issues this CTA's MMAs
    const int unit = blockIdx.x / ncta, nunits = gridDim.x / ncta;
    const int k0 = CG == 2 ? 0 : rank * p.per, k1 = min(p.nk, k0 + p.per);
    unsigned char* out_smem = smem + p.stages * p.stage_bytes;
    unsigned char* sf_smem = out_smem + (CG == 2 ? kOutBytes : 0);
    const int sf_slot_bytes = kSfBytes * (1 + NSUB * p.sf_blocks);
    // This cluster's tiles. Weight rows n0 .. n0 + rows - 1 of a CTA against row chunk rc of x. With one row chunk the
    // CTAs (CG = 1) share the weight rows evenly in units of 16 and end with a part of a tile: whole tiles would leave
    // SMs idle in the last round (128256 rows on 152 SMs: 7 rounds for 6.6 rounds' work).
    const bool even = CG == 1 && p.split == 1 && p.nrc == 1;
    const int parts = (p.N + kPartRows - 1) / kPartRows;
    const int r0 = even ? static_cast<int>(static_cast<int64_t>(parts) * unit / nunits) * kPartRows : 0;
    const int r1 = even ? static_cast<int>(static_cast<int64_t>(parts) * (unit + 1) / nunits) * kPartRows : 0;
    const int t0 = even ? 0 : unit, t1 = even ? (r1 - r0 + kTileN - 1) / kTileN : p.ntiles, dt = even ? 1 : nunits;
    struct Tile {
        int rc, n0, rows;
    };
    auto tile = [&](int t) -> Tile {
        if (even) return Tile{0, r0 + t * kTileN, min(kTileN, r1 - r0 - t * kTileN)};
        return Tile{t % p.nrc, (CG * (t / p.nrc) + (CG == 2 ? rank : 0)) * kTileN, kTileN};
    };

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&bar_full[s], 1);
            mbar_init(&bar_empty[s], 1);
        }
        for (int s = 0; s < kSfSlots; ++s) {
            mbar_init(&bar_sf_full[s], 32 * CG);
            mbar_init(&bar_sf_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar_acc_full[s], 1);
            mbar_init(&bar_acc_empty[s], kEpiWarps * CG);
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        if (CG == 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_holder)),
                         "r"(p.tmem_cols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_holder)),
                         "r"(p.tmem_cols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    if (ncta > 1) cg::this_cluster().sync();  // the other CTAs' barriers are there
    tc_fence_after();
    const uint32_t tmem = tmem_holder;
    if (warp == 0 && lane == 0) {
        // The first boxes of the weight on their way to L2 while an earlier kernel ends (a hint: what that kernel
        // writes to them still arrives)
        const Tile tl = tile(t0);
        for (int kc = k0; t0 < t1 && kc < min(k1, k0 + p.stages); ++kc) prefetch_box(&tm_w, kc * kStageK, tl.n0);
    }
    pdl_wait_prior();

    if (warp == 0) {
        // ------------------------------------------------------- loads ---
        const bool issue = elect_one();  // the warp goes through its loops together, one lane issues (see warp 1)
        const uint32_t full = smem_u32(bar_full), empty = smem_u32(bar_empty), smem0 = smem_u32(smem);
        const uint32_t full_at = CG == 2 ? cluster_addr(bar_full, 0) : full;
        const int xbox = p.Nr / CG;  // rows of x in a box
        uint32_t st = 0, phase = 1;  // stage and the parity of its last use (none yet: passes)
        bool ok = true;
        for (int t = t0; ok && t < t1; t += dt) {
            const Tile tl = tile(t);
            const int x0 = tl.rc * NSUB * p.Nr + (CG == 2 ? rank * xbox : 0);
            const uint32_t bytes = CG == 2 ? 2u * p.stage_bytes : static_cast<uint32_t>((tl.rows + p.Nr) * kStageK);
            for (int kc = k0; kc < k1; ++kc) {
                if (!wait_warp(empty + st * 8, phase)) {
                    ok = false;
                    break;
                }
                if (issue) {
                    const uint32_t dst = smem0 + st * p.stage_bytes, bar = full_at + st * 8;
                    if (rank == lead) mbar_arrive_expect_tx(&bar_full[st], bytes);
                    if (CG == 2 || tl.rows == kTileN) {
                        load_box<CG>(dst, &tm_w, kc * kStageK, tl.n0, bar);
                    } else {
                        for (int r = 0; r < tl.rows; r += kPartRows)
                            load_box<CG>(dst + r * kStageK, &tm_more, kc * kStageK, tl.n0 + r, bar);
                    }
#pragma unroll
                    for (int a = 0; a < NSUB; ++a)
                        load_box<CG>(dst + kWBytes + a * xbox * kStageK, &tm_x, kc * kStageK, x0 + a * p.Nr, bar);
                }
                if (++st == static_cast<uint32_t>(p.stages)) {
                    st = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok && issue) raise_status(p.status, kDevTimeout);
        // The CTA does not end before the MMAs that read its last stages, and their arrivals, are done. (Where a
        // wait has given up, the copies have had its limit, far more than they take.)
        for (int s = 0; ok && s < p.stages; ++s) {
            ok = wait_warp(empty + st * 8, phase);
            if (++st == static_cast<uint32_t>(p.stages)) {
                st = 0;
                phase ^= 1;
            }
        }
    } else if (warp == 1) {
        // -------------------------------------------------------- MMAs ---
        if (rank == lead) {
            // The warp goes through the loops together and one lane issues, so that descriptors, addresses and
            // the loops' conditions stay in uniform registers: a lane on its own took 720 clocks a stage, whatever
            // its MMAs' size, and 1050 with divisions for stage and parity (four MMAs of 224 rows take 448).
            const uint32_t idesc = idesc_mxf8(kTileN * CG, p.Nr);
            const bool issue = elect_one();
            const uint32_t full = smem_u32(bar_full), empty = smem_u32(bar_empty);
            const uint32_t sf_full = smem_u32(bar_sf_full), sf_empty = smem_u32(bar_sf_empty);
            const uint32_t acc_full = smem_u32(bar_acc_full), acc_empty = smem_u32(bar_acc_empty);
            uint32_t st = 0, phase = 0, slot = 0, sf_phase = 0;
            uint32_t buf = 0, acc_phase = 1;  // (NSUB = 1) the accumulator; the parity of its last reading (none yet: passes)
            const uint32_t base = ((smem_u32(smem) & 0x3FFFFu) >> 4) | (1u << 16);
            const uint64_t sf_base = sf_desc(smem_u32(sf_smem));
            const uint32_t step = static_cast<uint32_t>(p.stage_bytes) >> 4;
            const uint32_t x_step = static_cast<uint32_t>(p.Nr / CG * kStageK) >> 4;
            const uint32_t sfb_step = 4u * p.sf_blocks;
            uint32_t desc = base;
            bool ok = true;
            for (int t = t0; ok && t < t1; t += dt) {
                for (int kb = k0; ok && kb < k1; kb += p.chunk) {
                    const int ke = min(k1, kb + p.chunk);
                    for (int kg = kb; kg < ke; kg += kGroup) {
                        // The next group's scale words into this slot's columns. The slot was filled
                        // after the MMAs that read these columns last had ended.
                        const bool first = kg == kb, last = kg + kGroup >= ke;
                        if (!wait_warp<CG == 2>(sf_full + slot * 8, sf_phase) ||
                            (first && !wait_warp(acc_empty + buf * 8, acc_phase))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t sfa = tmem + p.sf_col + slot * p.sf_cols;
                        const uint64_t sd = sf_base + static_cast<uint32_t>(slot * sf_slot_bytes >> 4);
                        if (issue)
                            for (int b = 0; b <= NSUB * p.sf_blocks; ++b) copy_sf<CG>(sfa + 4 * b, sd + b * (kSfBytes >> 4));
                        const uint32_t d = tmem + buf * p.acc_stride;
                        // A stage's MMAs of accumulator a (K = 32 each: 32 bytes along the swizzled row)
                        auto mmas = [&](int i, int a, uint32_t aw) {
                            const uint32_t id = idesc | (static_cast<uint32_t>(i) << 4) | (static_cast<uint32_t>(i) << 29);
                            const uint32_t ax = aw + (kWBytes >> 4) + a * x_step;
#pragma unroll
                            for (int kk = 0; kk < kStageK / 32; ++kk)
                                mma_mxf8<CG>(d + a * p.acc_stride, aw + 2 * kk, ax + 2 * kk, id, sfa, sfa + 4 + a * sfb_step,
                                             i > 0 || kk > 0 ? 1 : !first);
                        };
                        // Two accumulators take turns stage by stage; at a sum's ends the group goes through
                        // the first and then the second, so that each is read while the other is summed (a
                        // group of 2 x 224 rows: 1800 clocks each).
                        const bool apart = NSUB == 2 && (first || last) && kg + kGroup <= ke;
                        const uint32_t desc0 = desc, st0 = st;
#pragma unroll
                        for (int i = 0; i < kGroup; ++i) {
                            if (kg + i >= ke) break;
                            if (!wait_warp(full + st * 8, phase)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            if (issue) mmas(i, 0, desc);
                            if (!apart) {
                                if (NSUB == 2) {
                                    if (i == 0 && first) {  // the second accumulator's last sums have been read
                                        if (!wait_warp(acc_empty + 8, acc_phase)) {
                                            ok = false;
                                            break;
                                        }
                                        tc_fence_after();
                                    }
                                    if (issue) mmas(i, 1, desc);
                                }
                                if (issue) commit<CG>(empty + st * 8);
                            }
                            desc += step;
                            if (++st == static_cast<uint32_t>(p.stages)) {
                                st = 0;
                                phase ^= 1;
                                desc = base;
                            }
                        }
                        if (!ok) break;
                        if (last && issue) commit<CG>(acc_full + buf * 8);
                        if (NSUB == 2) {
                            if (apart) {
                                if (first && !wait_warp(acc_empty + 8, acc_phase)) {
                                    ok = false;
                                    break;
                                }
                                tc_fence_after();
                                uint32_t da = desc0, sa = st0;
#pragma unroll
                                for (int i = 0; i < kGroup; ++i) {
                                    if (issue) {
                                        mmas(i, 1, da);
                                        commit<CG>(empty + sa * 8);
                                    }
                                    da += step;
                                    if (++sa == static_cast<uint32_t>(p.stages)) {
                                        sa = 0;
                                        da = base;
                                    }
                                }
                            }
                            if (last && issue) commit<CG>(acc_full + 8);
                        }
                        if (issue) commit<CG>(sf_empty + slot * 8);
                        if (++slot == kSfSlots) {
                            slot = 0;
                            sf_phase ^= 1;
                        }
                    }
                    if (NSUB == 2) {
                        acc_phase ^= 1;
                    } else {
                        buf ^= 1;
                        if (buf == 0) acc_phase ^= 1;
                    }
                }
            }
            if (!ok && issue) raise_status(p.status, kDevTimeout);
        }
    } else if (warp == 2) {
        // ------------------------------------------------------ scales ---
        const uint32_t sf_empty = smem_u32(bar_sf_empty), sf_full = cluster_addr(bar_sf_full, lead);
        uint32_t slot = 0, sf_phase = 1;
        bool ok = true;
        constexpr int kBlocks = 2 * NSUB;  // 128-row blocks of x at most
        constexpr int kWRows = CG == 1 ? 4 : 1;  // (a part's rows may lie in two of the weight's blocks)
        const int g0 = k0 / kGroup, g1 = (k1 + kGroup - 1) / kGroup;
        uint32_t ww[kWRows], xw[kBlocks][4];
        const uint32_t* wrow[kWRows];
        int m0 = 0, tf = t0, gf = g0;  // the next words to fetch: tile and group
        auto rows_of = [&](int t) {
            const Tile tl = tile(t);
            m0 = tl.rc * NSUB * p.Nr;
#pragma unroll
            for (int i = 0; i < kWRows; ++i)
                wrow[i] = p.w_scales + static_cast<size_t>(min((tl.n0 + (CG == 1 ? i * 32 + lane : 0)) / kTileN, p.nwt - 1)) * p.sf_row_words;
        };
        // The next words are on their way while the slots are full, those of the next tile too (640 rows of zeros against
        // 128256 x 4096: 201 us, 193 with it). No condition on a load, which would be waited for where the two cases
        // meet (10 rows against 128256 x 8192: 213 us, 180 without): rows past x's end take its last row's scales (their
        // codes are zeros, their outputs are not stored), and behind the last tile its first words come again.
        auto fetch = [&]() {
#pragma unroll
            for (int i = 0; i < kWRows; ++i) ww[i] = ld_prior(wrow[i] + gf);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int a = NSUB == 2 && b >= p.sf_blocks ? 1 : 0;  // the block's accumulator
                    const int m = min(m0 + a * p.Nr + (b - a * p.sf_blocks) * 128 + i * 32 + lane, p.M - 1);
                    xw[b][i] = ld_prior(p.x_scales + static_cast<size_t>(m) * p.sf_row_words + gf);
                }
            if (++gf == g1) {
                gf = g0;
                tf += dt;
                if (tf < t1) rows_of(tf);
            }
        };
        int left = t0 < t1 ? (t1 - t0 + dt - 1) / dt * (g1 - g0) : 0;
        if (left > 0) {
            rows_of(t0);
            fetch();
        }
        for (; left > 0; --left) {
            if (!wait_warp_sleep(sf_empty + slot * 8, sf_phase)) {
                ok = false;
                break;
            }
            const uint32_t dst = smem_u32(sf_smem + slot * sf_slot_bytes) + lane * 16;
            sts128(dst, CG == 1 ? make_uint4(ww[0], ww[kWRows / 4], ww[kWRows / 2], ww[kWRows - 1])
                                : make_uint4(ww[0], ww[0], ww[0], ww[0]));
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
                if (b < NSUB * p.sf_blocks) sts128(dst + (1 + b) * kSfBytes, make_uint4(xw[b][0], xw[b][1], xw[b][2], xw[b][3]));
            fence_proxy_async_smem();
            if (CG == 1 || rank == lead) mbar_arrive(&bar_sf_full[slot]);
            else arrive_at(sf_full + slot * 8);
            if (++slot == kSfSlots) {
                slot = 0;
                sf_phase ^= 1;
            }
            fetch();
        }
        if (!ok) raise_status(p.status, kDevTimeout);
        for (int s = 0; ok && s < kSfSlots; ++s) {
            ok = wait_warp_sleep(sf_empty + slot * 8, sf_phase);
            if (++slot == kSfSlots) {
                slot = 0;
                sf_phase ^= 1;
            }
        }
    } else if (warp >= 4) {
        // ---------------------------------------------------- epilogue ---
        // Lane quarter warp % 4; warps 4..7 read the first half of the columns, 8..11 the second
        const int q4 = warp & 3, half = (warp - 4) >> 2;
        const int b0 = half_first(p.Nr, half), nb = half_count(p.Nr, half);
        const uint32_t from = tmem + (static_cast<uint32_t>(q4 * 32) << 16) + b0 * 16;
        const uint32_t freed = cluster_addr(bar_acc_empty, lead), acc_full = smem_u32(bar_acc_full);
        uint32_t buf = 0, acc_phase = 0;
        bool ok = true;
        auto wait_full = [&](uint32_t b) -> bool {
            if (wait_warp_sleep(acc_full + b * 8, acc_phase)) {
                tc_fence_after();
                return true;
            }
            raise_status(p.status, kDevTimeout);
            return ok = false;
        };
        auto release = [&](uint32_t b) {  // the accumulator may take its next sums
            tc_fence_before();
            __syncwarp();
            if (lane != 0) return;
            if (CG == 1 || rank == lead) mbar_arrive(&bar_acc_empty[b]);
            else arrive_at_relaxed(freed + b * 8);  // (its loads have ended, nothing in memory goes with it)
        };
        auto next = [&]() {
            if (NSUB == 2) {
                acc_phase ^= 1;
            } else {
                buf ^= 1;
                if (buf == 0) acc_phase ^= 1;
            }
        };
        // (CG = 2) The way out, by each warp for its 32 columns: 16 rows at a time through one of its boxes in shared
        // memory, stored from there in bulk where the output's rows allow it
        constexpr int kBoxes = BF16 ? 4 : 2, kBoxBytes = kOutBytes / kEpiWarps / kBoxes;
        static_assert(kBoxBytes == 16 * 32 * (BF16 ? 2 : 4), "16 rows of 32 columns");
        const uint32_t box0 = smem_u32(out_smem) + (warp - 4) * (kOutBytes / kEpiWarps);
        uint32_t box = 0;
        auto box_free = [&]() {  // the box's last store has been read
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kBoxes - 1) : "memory");
            __syncwarp();
        };
        auto box_out = [&](int v0, int m, bool add) {
            const uint32_t at = box0 + box * kBoxBytes;
            if (p.bulk_out) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) store_block(&tm_more, at, v0, m, add);
                __syncwarp();
            } else if (v0 + lane < p.N) {
                // this lane's own column
                const int live = min(16, p.M - m);
                if (BF16) {
                    unsigned short* o = static_cast<unsigned short*>(p.out) + static_cast<size_t>(m) * p.N + v0 + lane;
                    for (int j = 0; j < live; ++j, o += p.N) {
                        unsigned short x;
                        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at + j * 64 + lane * 2) : "memory");
                        *o = x;
                    }
                } else {
                    float* o = static_cast<float*>(p.out) + static_cast<size_t>(m) * p.N + v0 + lane;
                    for (int j = 0; j < live; ++j, o += p.N) {
                        float x;
                        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at + j * 128 + lane * 4) : "memory");
                        *o = add ? *o + x : x;
                    }
                }
            }
            box = (box + 1) % kBoxes;
        };
        for (int t = t0; ok && t < t1; t += dt) {
            const Tile tl = tile(t);
            const int v0 = tl.n0 + q4 * 32, v = v0 + lane;
            const int row = tl.rc * NSUB * p.Nr + b0 * 16;
            if (CG == 2 && BF16) {
                // All accumulators are read, rounded and freed before the first store. (What does not fit in
                // registers here goes to L2, the shared memory leaves no L1: spills took as long as the MMAs.)
                uint32_t pk[NSUB][kHalfBlocks][8];
#pragma unroll
                for (int a = 0; a < NSUB; ++a) {
                    if (!ok || !wait_full(buf + a)) break;
#pragma unroll
                    for (int b = 0; b < kHalfBlocks; ++b) {
                        if (b < nb) {
                            float x[16];
                            tmem_ld16(from + (buf + a) * p.acc_stride + b * 16, x);
#pragma unroll
                            for (int j = 0; j < 8; ++j) pk[a][b][j] = pack2(x[2 * j], x[2 * j + 1]);
                        }
                    }
                    release(buf + a);
                }
                next();
                if (!ok) break;
#pragma unroll
                for (int a = 0; a < NSUB; ++a) {
#pragma unroll
                    for (int b = 0; b < kHalfBlocks; ++b) {
                        const int m = row + a * p.Nr + b * 16;
                        if (b < nb && m < p.M) {
                            box_free();
                            const uint32_t to = box0 + box * kBoxBytes + lane * 2;
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + j * 64),
                                             "h"(static_cast<unsigned short>((j & 1) ? pk[a][b][j >> 1] >> 16 : pk[a][b][j >> 1]))
                                             : "memory");
                            box_out(v0, m, false);
                        }
                    }
                }
            } else if (CG == 2) {
                for (int kb = k0; ok && kb < k1; kb += p.chunk, next()) {
                    // a later chunk's sums are added to the outputs, once their stores are there
                    const bool add = kb > k0;
                    if (add && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
#pragma unroll 1
                    for (int a = 0; a < NSUB; ++a) {
                        if (!wait_full(buf + a)) break;
                        float x[kHalfBlocks][16];
#pragma unroll
                        for (int b = 0; b < kHalfBlocks; ++b)
                            if (b < nb) tmem_ld16(from + (buf + a) * p.acc_stride + b * 16, x[b]);
                        release(buf + a);
#pragma unroll
                        for (int b = 0; b < kHalfBlocks; ++b) {
                            const int m = row + a * p.Nr + b * 16;
                            if (b < nb && m < p.M) {
                                box_free();
                                const uint32_t to = box0 + box * kBoxBytes + lane * 4;
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(to + j * 128), "f"(x[b][j]) : "memory");
                                box_out(v0, m, add);
                            }
                        }
                    }
                }
            } else {
                float acc[kHalfBlocks][16];
#pragma unroll
                for (int b = 0; b < kHalfBlocks; ++b)
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[b][j] = 0.0f;
                for (int kb = k0; ok && kb < k1; kb += p.chunk, next()) {
                    if (!wait_full(buf)) break;
#pragma unroll
                    for (int b = 0; b < kHalfBlocks; ++b) {
                        if (b >= nb) continue;
                        float x[16];
                        tmem_ld16(from + buf * p.acc_stride + b * 16, x);
#pragma unroll
                        for (int j = 0; j < 16; ++j) acc[b][j] += x[j];
                    }
                    release(buf);
                }
                if (!ok) break;
                const int live = min(nb * 16, p.M - row);  // rows of this warp (uniform, may be negative)
                if (p.split > 1) {
                    // Column j's partial sums of all ranks meet in CTA j % split: slot [j / split][rank][lane].
                    const uint32_t red = smem_u32(sf_smem + kSfSlots * sf_slot_bytes);
                    int slot = b0 * 16 / p.split, owner = b0 * 16 % p.split;
#pragma unroll
                    for (int b = 0; b < kHalfBlocks; ++b) {
                        if (b * 16 >= live) break;
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            if (b * 16 + j < live) {
                                const uint32_t at = red + ((slot * p.split + rank) * kTileN + q4 * 32 + lane) * 4;
                                uint32_t to;
                                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(owner));
                                store_remote(to, acc[b][j]);
                            }
                            if (++owner == p.split) {
                                owner = 0;
                                ++slot;
                            }
                        }
                    }
                } else if (v < min(p.N, tl.n0 + tl.rows)) {
                    const size_t at = static_cast<size_t>(row) * p.N + v;
#pragma unroll
                    for (int b = 0; b < kHalfBlocks; ++b) {
                        if (b * 16 >= live) continue;
                        const int64_t off = static_cast<int64_t>(b) * 16 * p.N;
                        if (BF16) store_rows(static_cast<__nv_bfloat16*>(p.out) + at + off, p.N, live - b * 16, acc[b]);
                        else store_rows(static_cast<float*>(p.out) + at + off, p.N, live - b * 16, acc[b]);
                    }
                }
            }
        }
        if (CG == 2 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    if (ncta > 1) cg::this_cluster().sync();
    tc_fence_after();
    if (CG == 1 && p.split > 1) {
        // One tile a cluster: the ranks' sums, in their order. A warp to a column, its loads side by side (128 threads
        // through the columns one after the other: 64 rows against 4096 x 4096 10.1 us, 3 of them here).
        const int rc = unit % p.nrc, v0 = (unit / p.nrc) * kTileN + lane;
        const float* red = reinterpret_cast<const float*>(sf_smem + kSfSlots * sf_slot_bytes) + lane;
        const int mn = min(p.Nr, p.M - rc * p.Nr);
        for (int s = warp; s * p.split + rank < mn; s += kLinThreads / 32) {
            const float* from = red + s * p.split * kTileN;
            float sum[kTileN / 32];
#pragma unroll
            for (int i = 0; i < kTileN / 32; ++i) sum[i] = 0.0f;
#pragma unroll
            for (int r = 0; r < kMaxSplit; ++r) {
                if (r >= p.split) break;
#pragma unroll
                for (int i = 0; i < kTileN / 32; ++i) sum[i] += from[r * kTileN + i * 32];
            }
            const size_t at = static_cast<size_t>(rc * p.Nr + s * p.split + rank) * p.N + v0;
#pragma unroll
            for (int i = 0; i < kTileN / 32; ++i) {
                if (v0 + i * 32 >= p.N) break;
                if (BF16) static_cast<__nv_bfloat16*>(p.out)[at + i * 32] = __float2bfloat16_rn(sum[i]);
                else static_cast<float*>(p.out)[at + i * 32] = sum[i];
            }
        }
        __syncwarp();
    }
    if (warp == 1) {
        if (CG == 1)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem_cols) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem_cols) : "memory");
    }
}

bool make_map(CUtensorMap* m, CUtensorMapDataType type, const void* base, uint64_t inner, uint64_t outer, uint64_t row_bytes,
              uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle) {
    auto fn = tensor_map_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {inner, outer};
    const cuuint64_t strides[1] = {row_bytes};
    const cuuint32_t box[2] = {box_inner, box_outer};
    const cuuint32_t estride[2] = {1, 1};
    return fn(m, type, 2, const_cast<void*>(base), dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool make_map_codes(CUtensorMap* m, const void* base, int inner, int outer, int box_outer) {
    return make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, static_cast<uint64_t>(inner), static_cast<uint64_t>(outer),
                    static_cast<uint64_t>(inner), kStageK, static_cast<uint32_t>(box_outer), CU_TENSOR_MAP_SWIZZLE_128B);
}

// SMs of the current device, asked once for each (calls of several threads may meet here).
int sm_count() {
    static std::atomic<int> known[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    std::atomic<int>& slot = known[dev % kMaxDevices];
    int n = slot.load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 1;
        slot.store(n, std::memory_order_relaxed);
    }
    return n;
}

// How many clusters of ncta CTAs run at once (GPCs hold no whole number of them), asked once for each size and
// device. A CTA has an SM for itself, whatever its share of the shared memory.
template <int CG, bool BF16>
cudaError_t clusters_at_once(int ncta, int* n) {
    *n = sm_count();
    if (ncta == 1) return cudaSuccess;
    static std::atomic<int> known[kMaxDevices][kMaxSplit + 1];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::atomic<int>& slot = known[dev % kMaxDevices][ncta];
    if ((*n = slot.load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    e = ensure_dyn_smem(reinterpret_cast<const void*>(linear_fp8_kernel<CG, BF16>), kSmemBudget);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ncta);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ncta));
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = kSmemBudget;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(n, linear_fp8_kernel<CG, BF16>, &cfg);
    if (e == cudaSuccess && *n > 0) slot.store(*n, std::memory_order_relaxed);
    return e;
}

int round_up(int x, int to) { return (x + to - 1) / to * to; }

template <int CG, bool BF16>
cudaError_t launch(LinParams& p, const void* x, const void* w, cudaStream_t stream) {
    constexpr int NSUB = CG;
    const int ncta = CG == 2 ? 2 : p.split;
    p.nrc = (p.M + p.Nr * NSUB - 1) / (p.Nr * NSUB);
    p.ntiles = p.nrc * ((p.nwt + CG - 1) / CG);
    p.stage_bytes = kWBytes + NSUB * (p.Nr / CG) * kStageK;
    p.sf_blocks = (p.Nr + 127) / 128;
    const int red_bytes = p.split > 1 ? (p.Nr + p.split) * kTileN * 4 : 0;
    const int sf_bytes = kSfSlots * kSfBytes * (1 + NSUB * p.sf_blocks);
    const int rest = 1024 + sf_bytes + red_bytes + (CG == 2 ? kOutBytes : 0);
    p.stages = std::min(kMaxStages, (kSmemBudget - rest) / p.stage_bytes);
    p.sf_row_words = fp8_scale_stride(p.K) / 4;
    p.acc_stride = static_cast<uint32_t>(round_up(p.Nr, 32));
    p.sf_col = 2 * p.acc_stride;
    p.sf_cols = 4u * (1 + NSUB * p.sf_blocks);
    p.tmem_cols = 32;
    while (p.tmem_cols < p.sf_col + kSfSlots * p.sf_cols) p.tmem_cols <<= 1;
    CUtensorMap tw, tx, to;
    if (!make_map_codes(&tw, w, p.K, p.N, kTileN) || !make_map_codes(&tx, x, p.K, p.M, p.Nr / CG)) return cudaErrorInvalidValue;
    constexpr int es = BF16 ? 2 : 4;
    p.bulk_out = CG == 2 && static_cast<int64_t>(p.N) * es % 16 == 0;
    if (p.bulk_out) {
        if (!make_map(&to, BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, p.out,
                      static_cast<uint64_t>(p.N), static_cast<uint64_t>(p.M), static_cast<uint64_t>(p.N) * es, 32, 16,
                      CU_TENSOR_MAP_SWIZZLE_NONE))
            return cudaErrorInvalidValue;
    } else if (!make_map_codes(&to, w, p.K, p.N, kPartRows)) {
        return cudaErrorInvalidValue;
    }
    const int smem = rest + p.stages * p.stage_bytes;
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(linear_fp8_kernel<CG, BF16>), smem);
    if (e != cudaSuccess) return e;
    int fit = 0;
    e = clusters_at_once<CG, BF16>(ncta, &fit);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    // A cluster that splits K has one tile. CTAs that share the weight's rows evenly have 16 rows at least, so that
    // fewer tiles than SMs still keep all of them busy (one tile a CTA / so, us: 10 rows against 10240 x 8192 24.9 /
    // 23.1, 100 rows against 12288 x 4096 17.1 / 16.0, 3 rows against 14336 x 4096 14.6 / 14.9).
    const int work = CG == 1 && p.split == 1 && p.nrc == 1 ? (p.N + kPartRows - 1) / kPartRows : p.ntiles;
    cfg.gridDim = dim3(static_cast<unsigned>((p.split > 1 ? p.ntiles : std::min(work, std::max(1, fit))) * ncta));
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ncta);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    count_launch();
    return cudaLaunchKernelEx(&cfg, linear_fp8_kernel<CG, BF16>, tw, tx, to, p);
}

template <bool BF16>
cudaError_t launch_dtype(int M, int N, int K, const void* x, const uint8_t* x_scales, const void* w,
                         const uint8_t* w_scales, void* out, int* status, cudaStream_t stream) {
    LinParams p{};
    p.M = M;
    p.N = N;
    p.K = K;
    p.nwt = (N + kTileN - 1) / kTileN;
    p.nk = (K + kStageK - 1) / kStageK;
    p.split = 1;
    p.per = round_up(p.nk, kGroup);
    p.x_scales = reinterpret_cast<const uint32_t*>(x_scales);
    p.w_scales = reinterpret_cast<const uint32_t*>(w_scales);
    p.out = out;
    p.status = status;
    const int sms = sm_count();
    const int subs = (M + kMaxNr - 1) / kMaxNr;
    const bool few = static_cast<long>(subs) * p.nwt * 2 <= sms;
    if (M > kMaxNr && !few) {
        // Pairs: the fewest accumulators of up to 224 rows, evenly, two of them to a tile. (What one accumulator holds is
        // for CTAs by themselves, which share the weight evenly: 224 rows against 128256 x 4096 110 us by pairs, 99;
        // 128 rows 109, 88.)
        const int per_row = round_up(subs, 2);
        p.Nr = round_up((M + per_row - 1) / per_row, 16);
        p.chunk = BF16 ? p.per : kF32Chunk2;
        return launch<2, BF16>(p, x, w, stream);
    }
    // Few tiles: 64 rows each while there are SMs for more than eight parts of K (500 rows against 512 x 4096: 7.5 us, 8.4
    // with 128), 128 else (200 against 2048 x 4096: 9.3 us with 64, 8.6; 90 against 6144 x 4096: 12.9, 10.5)
    const int max_rows = !few ? kMaxNr : (M + kMaxNrFew - 1) / kMaxNrFew * p.nwt * kMaxSplit <= sms ? 64 : kMaxNrFew;
    const int chunks = (M + max_rows - 1) / max_rows;
    p.Nr = round_up((M + chunks - 1) / chunks, 16);
    if (few) {
        // Few tiles: K split over clusters, one tile a cluster
        const int tiles = (M + p.Nr - 1) / p.Nr * p.nwt;
        const int groups = p.per / kGroup;
        int want = std::max(1, std::min({kMaxSplit, sms / tiles, groups}));
        for (int fit = 0; want > 1; --want) {
            const cudaError_t e = clusters_at_once<1, BF16>(want, &fit);
            if (e != cudaSuccess) return e;
            if (fit >= tiles) break;
        }
        p.per = (groups + want - 1) / want * kGroup;
        p.split = (groups * kGroup + p.per - 1) / p.per;
    }
    p.chunk = BF16 ? p.per : kF32Chunk1;
    return launch<1, BF16>(p, x, w, stream);
}

}  // namespace

cudaError_t launch_linear_fp8(int M, int N, int K, const void* x, const uint8_t* x_scales, const void* w,
                              const uint8_t* w_scales, int out_dtype, void* out, int* status, cudaStream_t stream) {
    // One row or two of a small weight: without the tensor cores' fixed cost. us, rows kernel / this one, on weights
    // that lie in L2: 1 row 512 x 2048 2.3 / 4.0, 4096 x 4096 4.7 / 5.9, 6144 x 4096 6.4 / 7.5, 8192 x 4096 8.9 / 7.9;
    // 2 rows 2048 x 4096 3.8 / 5.4, 4096 x 4096 5.9 / 5.9, 6144 x 4096 7.7 / 7.5, 8192 x 3584 11.7 / 7.6; on weights
    // that come from HBM: 1 row 2.1 / 4.1, 6.2 / 6.8, 8.3 / 8.2, 10.2 / 9.0; 2 rows 4.7 / 5.6, 7.3 / 6.9, 9.6 / 8.3,
    // 12.5 / 8.8.
    const int64_t weight = static_cast<int64_t>(N) * K;
    if ((M == 1 && weight <= 28 << 20) || (M == 2 && weight <= 17 << 20))
        return launch_linear_fp8_rows(M, N, K, x, x_scales, w, w_scales, out_dtype, out, stream);
    return out_dtype == 1 ? launch_dtype<true>(M, N, K, x, x_scales, w, w_scales, out, status, stream)
                          : launch_dtype<false>(M, N, K, x, x_scales, w, w_scales, out, status, stream);
}

}  // namespace eagle
