// Rows of 8-bit codes with a scale for each 128 entries (sm_103a):
// eagle_rmsnorm_fp8 (the residual's addition, the root-mean-square norm and the
// codes in one pass) and eagle_linear_fp8_pack (a weight's codes, one scale for
// each block of 128 x 128).
//
// A thread holds 16 neighbouring entries of a row in registers from the load to
// the codes, so a row is read once: the sum of squares goes over the row's
// threads (shuffles, then shared memory where a row has several warps), the
// largest |y| of a block of 128 over eight neighbouring lanes. A scale is the
// smallest power of two 2^k with amax <= 448 2^k, taken from amax's bits, and
// stored as the byte k + 127 that the block-scaled tensor instructions read.
// Sums are fp32: a thread's 16 squares in pairs, then a tree.

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "eagle_internal.cuh"
#include "quant_ptx.cuh"
#include "quant_ws.h"

namespace eagle {
namespace {

constexpr int kPer = 16;           // entries of a thread
constexpr int kNormThreads = 256;  // of a CTA, more where a row needs them

__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&v)[kPer]) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const uint4 u = ld_prior(reinterpret_cast<const uint4*>(p) + q);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[q * 8 + 2 * i] = __uint_as_float(w[i] << 16);
            v[q * 8 + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}
__device__ __forceinline__ void load16(const float* p, float (&v)[kPer]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint4 u = ld_prior(reinterpret_cast<const uint4*>(p) + q);
        v[4 * q] = __uint_as_float(u.x);
        v[4 * q + 1] = __uint_as_float(u.y);
        v[4 * q + 2] = __uint_as_float(u.z);
        v[4 * q + 3] = __uint_as_float(u.w);
    }
}
// v rounded to the rows' type, stored, and kept as rounded.
__device__ __forceinline__ void store16(__nv_bfloat16* p, float (&v)[kPer]) {
    uint32_t w[kPer / 2];
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    if (p == nullptr) return;
#pragma unroll
    for (int q = 0; q < 2; ++q) reinterpret_cast<uint4*>(p)[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
}
__device__ __forceinline__ void store16(float* p, float (&v)[kPer]) {
    if (p == nullptr) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) reinterpret_cast<float4*>(p)[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
}

// Scale byte of a block whose largest |y| has these bits; 0 where it is an infinity or NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    const int e = static_cast<int>(amax >> 23);
    if (e == 255) return 0u;
    return static_cast<uint32_t>(max(1, e - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0)));
}
// 16 codes of y under a scale byte (0: the block has no scale, its codes are NaN).
__device__ __forceinline__ uint4 codes16(const float (&y)[kPer], uint32_t byte) {
    if (byte == 0u) return make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
    const float inv = __uint_as_float((254u - byte) << 23);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i] * inv, y[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i + 2] * inv, y[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint32_t amax_bits(const float (&y)[kPer]) {
    uint32_t a = 0u;
#pragma unroll
    for (int i = 0; i < kPer; ++i) a = max(a, __float_as_uint(y[i]) & 0x7fffffffu);
    return a;
}

// The sum of a value over the wpr warps of a row; every thread of the CTA takes part.
__device__ __forceinline__ float row_sum(float v, int wpr, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (wpr == 1) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, first = warp / wpr * wpr;
    __syncthreads();  // the last use of red is over
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = lane < wpr ? red[first + lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename T>
__global__ void __launch_bounds__(1024) rmsnorm_fp8_kernel(RmsnormFp8Args a, int wpr) {
    __shared__ float red[32];
    __shared__ int odd;
    const int tid = threadIdx.x, warp = tid >> 5;
    const int rpc = (blockDim.x >> 5) / wpr;  // rows of a CTA
    const int row = blockIdx.x * rpc + warp / wpr;
    const int at = (tid - warp / wpr * wpr * 32) * kPer;  // this thread's first entry
    const bool live = row < a.rows && at < a.dim;
    pdl_launch_dependents();
    if (tid == 0) odd = 0;
    float w[kPer];
    pdl_wait_prior();
    float s[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) s[i] = 0.0f;
    const size_t off = static_cast<size_t>(row) * a.row_stride + at;
    if (live) {
        load16(static_cast<const T*>(a.x) + off, s);
        if (a.residual) {
            float r[kPer];
            load16(static_cast<const T*>(a.residual) + off, r);
#pragma unroll
            for (int i = 0; i < kPer; ++i) s[i] += r[i];
            store16(a.sum ? static_cast<T*>(a.sum) + off : static_cast<T*>(nullptr), s);
        }
        if (a.weight) load16(static_cast<const T*>(a.weight) + at, w);
    }
    if (a.weight) {  // uniform
        float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kPer; ++i) t[i & 3] = fmaf(s[i], s[i], t[i & 3]);
        const float n = static_cast<float>(a.dim);
        const float sq = row_sum((t[0] + t[1]) + (t[2] + t[3]), wpr, red);
        float rstd = 1.0f / sqrtf(sq / n + a.eps);
        // A row whose squares leave fp32's range has them summed at 2^-160 (eps does not count
        // then); one that holds an infinity or NaN has no norm.
        const bool far = !(sq <= 3.0e38f);
        if (wpr > 1 || __any_sync(0xffffffffu, far)) {
            if (wpr > 1) {
                if (far) odd = 1;
                __syncthreads();
            }
            if (wpr == 1 || odd) {
                constexpr float kDown = 0x1p-80f;
#pragma unroll
                for (int i = 0; i < 4; ++i) t[i] = 0.0f;
#pragma unroll
                for (int i = 0; i < kPer; ++i) t[i & 3] = fmaf(s[i] * kDown, s[i] * kDown, t[i & 3]);
                const float low = row_sum((t[0] + t[1]) + (t[2] + t[3]), wpr, red);
                if (far) {
                    rstd = low <= 3.0e38f ? 1.0f / sqrtf(low / n) : NAN;  // of the row at 2^-80
#pragma unroll
                    for (int i = 0; i < kPer; ++i) s[i] = s[i] * rstd * kDown;
                    rstd = 1.0f;
                }
            }
        }
        if (live) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) s[i] = s[i] * rstd * w[i];
        }
    }
    uint32_t amax = live ? amax_bits(s) : 0u;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (row >= a.rows) return;
    const uint32_t byte = scale_byte(amax);
    if (live) *reinterpret_cast<uint4*>(static_cast<char*>(a.codes) + static_cast<size_t>(row) * a.dim + at) = codes16(s, byte);
    if ((tid & 7) == 0) {
        const int block = at / kFp8Block;
        // the row's scales are filled up with zeros; where they reach past the row's threads, its last group writes them
        const int nb = (a.dim + kFp8Block - 1) / kFp8Block;
        uint8_t* out = a.scales + static_cast<size_t>(row) * a.scale_stride;
        if (block < nb) {
            out[block] = static_cast<uint8_t>(byte ? byte : 127u);
            if (byte == 0u) raise_status(a.status, kDevNonFinite);
            if (block == nb - 1)
                for (int b = nb; b < a.scale_stride; ++b) out[b] = 0;
        }
    }
}

// One CTA of 256 threads for each block of 128 x 128: two threads a row, 64 entries each.
__global__ void __launch_bounds__(256) fp8_pack_kernel(int N, int K, int scale_stride, const __nv_bfloat16* weight,
                                                       uint8_t* codes, uint8_t* scales) {
    __shared__ uint32_t red[8];
    const int tid = threadIdx.x;
    const int row = blockIdx.y * kFp8Block + tid / 2, col = blockIdx.x * kFp8Block + (tid & 1) * 64;
    pdl_launch_dependents();
    pdl_wait_prior();
    float y[4][kPer];
    uint32_t amax = 0u;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const bool live = row < N && col + q * kPer < K;
        if (live) {
            load16(weight + static_cast<size_t>(row) * K + col + q * kPer, y[q]);
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) y[q][i] = 0.0f;
        }
        amax = max(amax, amax_bits(y[q]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((tid & 31) == 0) red[tid >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, red[i]);
    const uint32_t byte = scale_byte(amax);
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (row < N && col + q * kPer < K)
            *reinterpret_cast<uint4*>(codes + static_cast<size_t>(row) * K + col + q * kPer) = codes16(y[q], byte);
    if (tid == 0) {
        uint8_t* out = scales + static_cast<size_t>(blockIdx.y) * scale_stride;
        out[blockIdx.x] = static_cast<uint8_t>(byte ? byte : 127u);
        if (blockIdx.x == gridDim.x - 1)
            for (int b = gridDim.x; b < scale_stride; ++b) out[b] = 0;
    }
}

}  // namespace

cudaError_t launch_rmsnorm_fp8(const RmsnormFp8Args& a, int dtype, cudaStream_t stream) {
    // warps of a row: one for 512 entries, and so many rows that a CTA has kNormThreads
    const int wpr = (a.dim + 32 * kPer - 1) / (32 * kPer);
    const int rpc = std::max(1, kNormThreads / 32 / wpr);
    const dim3 grid(static_cast<unsigned>((a.rows + rpc - 1) / rpc)), block(static_cast<unsigned>(wpr * rpc * 32));
    if (dtype == 1) return launch_pdl(rmsnorm_fp8_kernel<__nv_bfloat16>, grid, block, 0, stream, a, wpr);
    return launch_pdl(rmsnorm_fp8_kernel<float>, grid, block, 0, stream, a, wpr);
}

cudaError_t launch_fp8_pack(int N, int K, int scale_stride, const void* weight, void* codes, uint8_t* scales,
                            cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>((K + kFp8Block - 1) / kFp8Block), static_cast<unsigned>((N + kFp8Block - 1) / kFp8Block));
    return launch_pdl(fp8_pack_kernel, grid, dim3(256), 0, stream, N, K, scale_stride,
                      static_cast<const __nv_bfloat16*>(weight), static_cast<uint8_t*>(codes), scales);
}

}  // namespace eagle
