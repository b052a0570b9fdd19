// eagle_linear_fp8 for one row of x or two, without the tensor cores (sm_103a).
//
// The tensor-core kernel (k_linear_fp8.cu) has a fixed cost of some 4 us
// (tensor memory, TMA descriptors, the pipeline's ends, a cluster's exchange);
// a projection's weight for a single token streams in less. Here a warp holds
// 512 neighbouring codes of x (16 a lane, as fp32 values) and goes down the
// CTA's weight rows, 512 bytes of a row at a time, so a CTA of eight warps reads
// whole rows of 4096 codes; the warps' sums meet in shared memory. A lane's 16
// codes lie in one block of 128: their products are added as the codes' own
// values and scaled once, by the sum of the two exponents (in two halves, so
// that no intermediate leaves fp32's range before the product does).
//
// Bound by HBM, and by the conversions: 8 instructions to two 16-bit values, 16
// to fp32 ones for 16 codes, beside 8 M packed multiply-adds.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "eagle_internal.cuh"
#include "eagle_ws.h"
#include "quant_ptx.cuh"
#include "quant_ws.h"

namespace eagle {
namespace {

constexpr int kMaxWarps = 8;
constexpr int kSmWarps = 16;  // of an SM, at 128 registers a thread
constexpr int kChunk = 512;   // codes of K that a warp holds

struct RowsParams {
    int N, K, scale_stride, units;  // units of RG weight rows
    const uint8_t *x, *x_scales, *w, *w_scales;
    void* out;
    int out_bf16;
};

// 16 codes as fp32 pairs.
__device__ __forceinline__ void decode16(const uint4& u, uint64_t (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t two;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(two) : "h"(static_cast<unsigned short>(h ? w[i] >> 16 : w[i])));
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two));
            v[2 * i + h] = f2_pack(f.x, f.y);
        }
    }
}
// 2^e, e = -127 .. 127 (-127 is subnormal).
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(e < -126 ? 0x00400000u : static_cast<uint32_t>(e + 127) << 23); }

// M rows of x, RG weight rows at a time.
template <int M, int RG>
__global__ void __launch_bounds__(kMaxWarps * 32, 2) linear_fp8_rows_kernel(RowsParams p) {
    extern __shared__ float sums[];  // [warp][row of the CTA][M]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, threads = blockDim.x, warps = threads >> 5;
    const int u0 = static_cast<int>(static_cast<int64_t>(p.units) * blockIdx.x / gridDim.x);
    const int u1 = static_cast<int>(static_cast<int64_t>(p.units) * (blockIdx.x + 1) / gridDim.x);
    const int rows = (u1 - u0) * RG;
    pdl_launch_dependents();
    pdl_wait_prior();
    float* mine = sums + warp * rows * M;
    constexpr int V = RG * M;  // sums of a group
    for (int c = warp; c * kChunk < p.K; c += warps) {  // (no more warps than chunks)
        const int k = c * kChunk + lane * 16;
        const bool in = k < p.K;
        const uint8_t* at = p.w + static_cast<int64_t>(u0) * RG * p.K + k;
        const uint8_t* sc = p.w_scales + k / kFp8Block;
        auto fetch = [&](int u, uint4 (&to)[RG], int& e) {
#pragma unroll
            for (int r = 0; r < RG; ++r)
                to[r] = in && u * RG + r < p.N ? ld_prior(reinterpret_cast<const uint4*>(at + static_cast<int64_t>((u - u0) * RG + r) * p.K))
                                               : make_uint4(0u, 0u, 0u, 0u);
            e = in ? static_cast<int>(ld_prior(sc + static_cast<int64_t>(min(u * RG, p.N - 1) / kFp8Block) * p.scale_stride)) : 127;
        };
        uint4 cur[RG], nxt[RG];
        int e_cur = 127, e_nxt = 127;
        if (u0 < u1) fetch(u0, cur, e_cur);
        uint64_t x[M][8];
        int xe[M];
#pragma unroll
        for (int m = 0; m < M; ++m) {
            decode16(in ? ld_prior(reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(m) * p.K + k)) : make_uint4(0u, 0u, 0u, 0u), x[m]);
            xe[m] = in ? static_cast<int>(ld_prior(p.x_scales + static_cast<int64_t>(m) * p.scale_stride + k / kFp8Block)) : 127;
        }
        for (int u = u0; u < u1; ++u) {
            if (u + 1 < u1) fetch(u + 1, nxt, e_nxt);
            float scale[M][2];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const int e = xe[m] + e_cur - 254, h = e >> 1;  // exponents -254 .. 254 (255 is NaN)
                const bool nan = xe[m] == 255 || e_cur == 255;
                scale[m][0] = nan ? NAN : pow2(h);
                scale[m][1] = nan ? NAN : pow2(e - h);
            }
            float v[V];
#pragma unroll
            for (int r = 0; r < RG; ++r) {
                uint64_t w[8];
                decode16(cur[r], w);
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    uint64_t s0 = f2_mul(w[0], x[m][0]), s1 = f2_mul(w[1], x[m][1]);
#pragma unroll
                    for (int i = 2; i < 8; i += 2) {
                        s0 = f2_fma(w[i], x[m][i], s0);
                        s1 = f2_fma(w[i + 1], x[m][i + 1], s1);
                    }
                    const uint64_t s = f2_add(s0, s1);
                    v[r * M + m] = (f2_lo(s) + f2_hi(s)) * scale[m][0] * scale[m][1];
                }
            }
            // V sums over the warp: at each of the first steps a lane hands half of its values on
            int own = 0;
#pragma unroll
            for (int n = V / 2, o = 16; n >= 1; n >>= 1, o >>= 1) {
                const bool up = (lane & o) != 0;
                own = own * 2 + (up ? 1 : 0);
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
            }
#pragma unroll
            for (int o = 16 / V; o >= 1; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
            if ((lane & (32 / V - 1)) == 0) {
                float* to = mine + (u - u0) * V + own;
                *to = c == warp ? v[0] : *to + v[0];
            }
#pragma unroll
            for (int r = 0; r < RG; ++r) cur[r] = nxt[r];
            e_cur = e_nxt;
        }
    }
    __syncthreads();
    for (int i = tid; i < rows * M; i += threads) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kMaxWarps; ++w)
            if (w < warps) s += sums[w * rows * M + i];
        const int n = u0 * RG + i / M, m = i % M;
        if (n >= p.N) continue;
        const int64_t at = static_cast<int64_t>(m) * p.N + n;
        if (p.out_bf16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(s);
        else static_cast<float*>(p.out)[at] = s;
    }
}

template <int M, int RG>
cudaError_t launch(RowsParams& p, cudaStream_t stream) {
    p.units = (p.N + RG - 1) / RG;
    // the warps of a CTA that keep most of an SM's warps at work, all with the same number of chunks if they can
    const int chunks = (p.K + kChunk - 1) / kChunk;
    int warps = 1, best = 0;
    for (int n = 1; n <= std::min(kMaxWarps, chunks); ++n) {
        const int busy = kSmWarps / n * n * 1000 * chunks / ((chunks + n - 1) / n * n);
        if (busy >= best) {
            best = busy;
            warps = n;
        }
    }
    // as many CTAs as run at once, more where their rows' sums would not fit in shared memory beside one another
    const int ctas = kSmWarps / warps;
    const int most = 200 * 1024 / ctas / (warps * RG * M * 4);  // units of a CTA
    const int grid = std::max(std::min(p.units, 152 * ctas), (p.units + most - 1) / most);
    const int smem = (p.units + grid - 1) / grid * RG * M * warps * 4;
    const cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(linear_fp8_rows_kernel<M, RG>), smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(linear_fp8_rows_kernel<M, RG>, dim3(static_cast<unsigned>(grid)), dim3(static_cast<unsigned>(warps * 32)), static_cast<size_t>(smem),
                      stream, p);
}

}  // namespace

cudaError_t launch_linear_fp8_rows(int M, int N, int K, const void* x, const uint8_t* x_scales, const void* w,
                                   const uint8_t* w_scales, int out_dtype, void* out, cudaStream_t stream) {
    RowsParams p{N, K, fp8_scale_stride(K), 0, static_cast<const uint8_t*>(x), x_scales, static_cast<const uint8_t*>(w), w_scales,
                 out, out_dtype == 1};
    return M == 1 ? launch<1, 8>(p, stream) : launch<2, 4>(p, stream);
}

}  // namespace eagle
