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
//   tile (vt, rc)   weight rows 128 vt .. against rows Nr rc .. of x, summed
//                   over K in stages of 128 codes (128-byte rows, 128B swizzle)
//   warp 0          one lane streams the boxes of w and x into a ring (TMA)
//   warp 1          one lane issues the MMAs into an fp32 accumulator in tensor
//                   memory, double buffered across tiles, and the copies of the
//                   scale words into tensor memory (tcgen05.cp)
//   warp 2          lays the scale words out for those copies, one group of
//                   K = 512 after the other
//   warps 4..7      read the accumulator and store the outputs
// Rows and columns past the operands' ends arrive as zeros and are not stored.

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "eagle_ws.h"
#include "quant_ptx.cuh"
#include "quant_ws.h"
#include "tc_ptx.cuh"

namespace eagle {
namespace {

constexpr int kTileN = 128;   // weight rows of a tile (MMA M)
constexpr int kStageK = 128;  // codes of K of a stage
constexpr int kMaxNr = 224;   // rows of x of a tile (MMA N): two accumulators and the scales fit in 512 columns
constexpr int kMaxStages = 12;
constexpr int kSfSlots = 4;   // groups of scale words (K = 512) on their way
constexpr int kSfBytes = 512; // scale words of 128 rows and K = 512
constexpr int kLinThreads = 256;
constexpr int kWBytes = kTileN * kStageK;
constexpr int kSmemBudget = 224 * 1024;

struct LinParams {
    int M, N, K;
    int Nr, nrc;      // rows of x of a tile, row chunks
    int ntiles;
    int nk, ngroups;  // stages and groups of scale words of a tile
    int stages, stage_bytes;
    int sf_blocks;    // 128-row blocks of x scale words of a tile
    int sf_row_words; // scale words of a row
    uint32_t acc_stride, sf_col, sf_cols, tmem_cols;
    int out_bf16;
    const uint32_t *x_scales, *w_scales;
    void* out;
    int* status;
};

// Instruction descriptor of kind::mxf8f6f4: A and B e4m3 (0), both K-major, N >> 3 at bits 17-22,
// E8M0 scales (bit 23), M >> 4 at bits 24-28; the scale word's byte for B at bits 4-5, for A at 29-30.
__host__ __device__ constexpr uint32_t idesc_mxf8(int M, int N) {
    return (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void mma_mxf8(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, int accum) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(tmem_d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accum)
        : "memory");
}
// Descriptor of 32 rows of 16 bytes, one after the other (no swizzle): 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t sf_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 16) |
           (static_cast<uint64_t>(128 >> 4) << 32) | (1ull << 46);
}
// Those 512 bytes into four columns of tensor memory, the same in each quarter of its lanes.
__device__ __forceinline__ void copy_sf(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

__global__ void __launch_bounds__(kLinThreads, 1)
    linear_fp8_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                      const LinParams p) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ __align__(8) uint64_t bar_full[kMaxStages], bar_empty[kMaxStages], bar_sf_full[kSfSlots],
        bar_sf_empty[kSfSlots], bar_acc_full[2], bar_acc_empty[2];
    __shared__ uint32_t tmem_holder;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned char* sf_smem = smem + p.stages * p.stage_bytes;
    const int sf_slot_bytes = kSfBytes * (1 + p.sf_blocks);

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&bar_full[s], 1);
            mbar_init(&bar_empty[s], 1);
        }
        for (int s = 0; s < kSfSlots; ++s) {
            mbar_init(&bar_sf_full[s], 32);
            mbar_init(&bar_sf_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar_acc_full[s], 1);
            mbar_init(&bar_acc_empty[s], 128);
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_holder)),
                     "r"(p.tmem_cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_holder;
    pdl_wait_prior();

    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int t = blockIdx.x; ok && t < p.ntiles; t += gridDim.x) {
                const int rc = t % p.nrc, vt = t / p.nrc;
                for (int kc = 0; kc < p.nk; ++kc, ++it) {
                    const uint32_t st = it % p.stages;
                    if (it >= static_cast<uint32_t>(p.stages) &&
                        !mbar_wait_sleep(&bar_empty[st], ((it / p.stages) - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    unsigned char* dst = smem + st * p.stage_bytes;
                    mbar_arrive_expect_tx(&bar_full[st], p.stage_bytes);
                    tma_load_2d(dst, &tm_w, kc * kStageK, vt * kTileN, &bar_full[st]);
                    tma_load_2d(dst + kWBytes, &tm_x, kc * kStageK, rc * p.Nr, &bar_full[st]);
                }
            }
            if (!ok) raise_status(p.status, kDevTimeout);
            // the CTA does not end before its copies have arrived
            for (uint32_t i = it > static_cast<uint32_t>(p.stages) ? it - p.stages : 0u; i < it; ++i)
                if (!mbar_wait_sleep(&bar_full[i % p.stages], (i / p.stages) & 1)) break;
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = idesc_mxf8(kTileN, p.Nr);
            uint32_t it = 0, gr = 0;
            bool ok = true;
            int lt = 0;
            for (int t = blockIdx.x; ok && t < p.ntiles; t += gridDim.x, ++lt) {
                const int buf = lt & 1;
                if (lt >= 2 && !mbar_wait_sleep(&bar_acc_empty[buf], ((lt >> 1) - 1) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + buf * p.acc_stride;
                uint32_t sfa = 0, sfb = 0;
                for (int kc = 0; kc < p.nk; ++kc, ++it) {
                    if ((kc & 3) == 0) {
                        // The next group's scale words into this slot's columns. The slot was filled
                        // after the MMAs that read these columns last had ended.
                        const uint32_t slot = gr % kSfSlots;
                        if (!mbar_wait_sleep(&bar_sf_full[slot], (gr / kSfSlots) & 1)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t src = smem_u32(sf_smem + slot * sf_slot_bytes);
                        sfa = tmem + p.sf_col + slot * p.sf_cols;
                        sfb = sfa + 4;
                        for (int b = 0; b <= p.sf_blocks; ++b) copy_sf(sfa + 4 * b, sf_desc(src + b * kSfBytes));
                    }
                    const uint32_t st = it % p.stages;
                    if (!mbar_wait_sleep(&bar_full[st], (it / p.stages) & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t aW = smem_u32(smem + st * p.stage_bytes);
                    const uint32_t aX = aW + kWBytes;
                    const uint32_t id = idesc | (static_cast<uint32_t>(kc & 3) << 4) | (static_cast<uint32_t>(kc & 3) << 29);
#pragma unroll
                    for (int kk = 0; kk < kStageK / 32; ++kk)  // K = 32 per MMA: 32 bytes along the swizzled row
                        mma_mxf8(d, smem_desc(aW + kk * 32, 16, 1024), smem_desc(aX + kk * 32, 16, 1024), id, sfa, sfb,
                                 (kc > 0 || kk > 0) ? 1 : 0);
                    mma_commit(&bar_empty[st]);
                    if ((kc & 3) == 3 || kc == p.nk - 1) {
                        mma_commit(&bar_sf_empty[gr % kSfSlots]);
                        ++gr;
                    }
                }
                if (ok) mma_commit(&bar_acc_full[buf]);
            }
            if (!ok) raise_status(p.status, kDevTimeout);
        }
        __syncwarp();
    } else if (warp == 2) {
        uint32_t gr = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < p.ntiles; t += gridDim.x) {
            const int rc = t % p.nrc, vt = t / p.nrc;
            const int m0 = rc * p.Nr, mn = min(p.Nr, p.M - m0);
            for (int g = 0; g < p.ngroups; ++g, ++gr) {
                const uint32_t slot = gr % kSfSlots;
                const uint32_t ww = ld_prior(p.w_scales + static_cast<size_t>(vt) * p.sf_row_words + g);
                uint32_t xw[2][4];
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = b * 128 + i * 32 + lane;
                        xw[b][i] = r < mn ? ld_prior(p.x_scales + static_cast<size_t>(m0 + r) * p.sf_row_words + g) : 0u;
                    }
                if (gr >= kSfSlots && !__all_sync(0xffffffffu, mbar_wait_sleep(&bar_sf_empty[slot], ((gr / kSfSlots) - 1) & 1))) {
                    ok = false;
                    break;
                }
                const uint32_t dst = smem_u32(sf_smem + slot * sf_slot_bytes) + lane * 16;
                sts128(dst, make_uint4(ww, ww, ww, ww));
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    if (b < p.sf_blocks) sts128(dst + (1 + b) * kSfBytes, make_uint4(xw[b][0], xw[b][1], xw[b][2], xw[b][3]));
                fence_proxy_async_smem();
                mbar_arrive(&bar_sf_full[slot]);
            }
        }
        if (!ok) raise_status(p.status, kDevTimeout);
    } else if (warp >= 4) {
        const int q4 = warp & 3;
        const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
        int lt = 0;
        for (int t = blockIdx.x; t < p.ntiles; t += gridDim.x, ++lt) {
            const int rc = t % p.nrc, vt = t / p.nrc;
            const int buf = lt & 1;
            if (!__all_sync(0xffffffffu, mbar_wait_sleep(&bar_acc_full[buf], (lt >> 1) & 1))) {
                raise_status(p.status, kDevTimeout);
                break;
            }
            tc_fence_after();
            const int v = vt * kTileN + q4 * 32 + lane;
            const int m0 = rc * p.Nr;
            const int mn = min(p.Nr, p.M - m0);  // live rows of the chunk (uniform)
            const uint32_t cols = tmem + lane_off + buf * p.acc_stride;
            for (int c = 0; c < mn; c += 16) {
                float x[16];
                tmem_ld16(cols + c, x);
                if (v < p.N) {
                    const int jn = min(16, mn - c);
                    const size_t at = static_cast<size_t>(m0 + c) * p.N + v;
                    if (p.out_bf16) {
                        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + at;
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (j < jn) o[static_cast<size_t>(j) * p.N] = __float2bfloat16_rn(x[j]);
                    } else {
                        float* o = static_cast<float*>(p.out) + at;
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (j < jn) o[static_cast<size_t>(j) * p.N] = x[j];
                    }
                }
            }
            // the accumulator may take the tile after next
            tc_fence_before();
            mbar_arrive(&bar_acc_empty[buf]);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem_cols) : "memory");
}

bool make_map_codes(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint32_t box_outer) {
    auto fn = tensor_map_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {inner, outer};
    const cuuint64_t strides[1] = {inner};
    const cuuint32_t box[2] = {kStageK, box_outer};
    const cuuint32_t estride[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estride,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
    static int n = 0;
    if (n == 0) {
        int dev = 0;
        cudaGetDevice(&dev);
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (n <= 0) n = 1;
    }
    return n;
}

}  // namespace

cudaError_t launch_linear_fp8(int M, int N, int K, const void* x, const uint8_t* x_scales, const void* w,
                              const uint8_t* w_scales, int out_dtype, void* out, int* status, cudaStream_t stream) {
    LinParams p{};
    p.M = M;
    p.N = N;
    p.K = K;
    p.nrc = (M + kMaxNr - 1) / kMaxNr;
    const int per = (M + p.nrc - 1) / p.nrc;
    p.Nr = (per + 15) & ~15;
    p.ntiles = p.nrc * ((N + kTileN - 1) / kTileN);
    p.nk = (K + kStageK - 1) / kStageK;
    p.ngroups = (p.nk + 3) / 4;
    p.stage_bytes = kWBytes + (p.Nr * kStageK + 1023) / 1024 * 1024;
    p.sf_blocks = (p.Nr + 127) / 128;
    const int sf_bytes = kSfSlots * kSfBytes * (1 + p.sf_blocks);
    p.stages = std::min(kMaxStages, (kSmemBudget - 1024 - sf_bytes) / p.stage_bytes);
    p.sf_row_words = fp8_scale_stride(K) / 4;
    p.acc_stride = (static_cast<uint32_t>(p.Nr) + 31u) & ~31u;
    p.sf_col = 2 * p.acc_stride;
    p.sf_cols = 4u * (1 + p.sf_blocks);
    p.tmem_cols = 32;
    while (p.tmem_cols < p.sf_col + kSfSlots * p.sf_cols) p.tmem_cols <<= 1;
    p.out_bf16 = out_dtype == 1;
    p.x_scales = reinterpret_cast<const uint32_t*>(x_scales);
    p.w_scales = reinterpret_cast<const uint32_t*>(w_scales);
    p.out = out;
    p.status = status;
    CUtensorMap tw, tx;
    if (!make_map_codes(&tw, w, static_cast<uint64_t>(K), static_cast<uint64_t>(N), kTileN) ||
        !make_map_codes(&tx, x, static_cast<uint64_t>(K), static_cast<uint64_t>(M), static_cast<uint32_t>(p.Nr)))
        return cudaErrorInvalidValue;
    const int smem = p.stages * p.stage_bytes + sf_bytes + 1024;
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(linear_fp8_kernel), smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(linear_fp8_kernel, dim3(std::min(p.ntiles, sm_count())), dim3(kLinThreads),
                      static_cast<size_t>(smem), stream, tw, tx, p);
}

}  // namespace eagle
