// Rows of 8-bit codes with a scale for each 128 entries (sm_103a):
// eagle_rmsnorm_fp8 (the residual's addition, the root-mean-square norm and the
// codes in one pass) and eagle_linear_fp8_pack (a weight's codes, one scale for
// each block of 128 x 128).
//
// A thread holds 16 entries of a block of 128 (eight neighbouring lanes hold
// the block, each 16 bytes of 128 bytes that a load or store covers) in
// registers from the load to the codes, so a row is read once: the sum of
// squares goes over the row's threads (shuffles, then shared memory where a row
// has several warps, one barrier a row), the largest |y| of a block over its
// eight lanes. A scale is the smallest power of two 2^k with amax <= 448 2^k,
// taken from amax's bits, and stored as the byte k + 127 that the block-scaled
// tensor instructions read. Sums are fp32: a thread's 16 squares in four parts,
// then a tree.
//
// Bound by HBM, nearly so by instructions (a thread spends 370 to 480 on its part
// of a row). CTAs stay for several rows, so that the weight comes from L1, and
// load the next rows before they reduce one where registers allow it. Measured:
// 3904 bf16 rows of 5120 with a residual (140 MB) 25 us, 82% of HBM; 8001 fp32
// rows of 8192 without (328 MB) 55 us, 88%, with one (853 MB) 136 us, 92%; 8001
// bf16 rows of 8192 without (197 MB) 48 us, 60%, the instructions' time; 640 rows of
// 4096 5.2 us, 10 rows 2.1.

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>

#include "eagle_internal.cuh"
#include "quant_ptx.cuh"
#include "quant_ws.h"

namespace eagle {
namespace {

constexpr int kPer = 16;           // entries of a thread
constexpr int kNormThreads = 256;  // of a CTA, more where a row needs them

// The 16 entries of a thread as loaded: V vectors of 16 bytes.
template <typename T>
struct Raw {
    static constexpr int V = kPer * static_cast<int>(sizeof(T)) / 16, N = 16 / static_cast<int>(sizeof(T));
    uint4 u[V];
};
// Vector q of lane l (0..7) of a block: entries q * 8 N + l N ..
template <typename T>
__device__ __forceinline__ int vec_at(int q, int l) { return (q * 8 + l) * Raw<T>::N; }

template <typename T>
__device__ __forceinline__ void load16(const T* block, int l, int left, Raw<T>& r) {
    if (left >= kFp8Block) {
#pragma unroll
        for (int q = 0; q < Raw<T>::V; ++q) r.u[q] = ld_prior(reinterpret_cast<const uint4*>(block + vec_at<T>(q, l)));
        return;
    }
#pragma unroll
    for (int q = 0; q < Raw<T>::V; ++q)
        r.u[q] = vec_at<T>(q, l) < left ? ld_prior(reinterpret_cast<const uint4*>(block + vec_at<T>(q, l))) : make_uint4(0u, 0u, 0u, 0u);
}
// The 16 entries as eight packed pairs (two results an instruction).
__device__ __forceinline__ void unpack16(const Raw<__nv_bfloat16>& r, uint64_t (&v)[kPer / 2]) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const uint32_t w[4] = {r.u[q].x, r.u[q].y, r.u[q].z, r.u[q].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[q * 4 + i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
}
__device__ __forceinline__ void unpack16(const Raw<float>& r, uint64_t (&v)[kPer / 2]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v[2 * q] = f2_pack(__uint_as_float(r.u[q].x), __uint_as_float(r.u[q].y));
        v[2 * q + 1] = f2_pack(__uint_as_float(r.u[q].z), __uint_as_float(r.u[q].w));
    }
}
// v rounded to the rows' type, kept as rounded, and stored.
__device__ __forceinline__ void store16(__nv_bfloat16* block, int l, int left, uint64_t (&v)[kPer / 2]) {
    uint32_t w[kPer / 2];
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f2_lo(v[i]), f2_hi(v[i]));
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
        v[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
    if (block == nullptr) return;
#pragma unroll
    for (int q = 0; q < 2; ++q)
        if (vec_at<__nv_bfloat16>(q, l) < left)
            *reinterpret_cast<uint4*>(block + vec_at<__nv_bfloat16>(q, l)) = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
}
__device__ __forceinline__ void store16(float* block, int l, int left, uint64_t (&v)[kPer / 2]) {
    if (block == nullptr) return;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (vec_at<float>(q, l) < left)
            *reinterpret_cast<float4*>(block + vec_at<float>(q, l)) = make_float4(f2_lo(v[2 * q]), f2_hi(v[2 * q]), f2_lo(v[2 * q + 1]), f2_hi(v[2 * q + 1]));
}

// Scale byte of a block whose largest |y| has these bits; 0 where it is an infinity or NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    const int e = static_cast<int>(amax >> 23);
    if (e == 255) return 0u;
    return static_cast<uint32_t>(max(1, e - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0)));
}
// Four codes of y * inv; NaN for those of a block without a scale.
__device__ __forceinline__ uint32_t codes4(const uint64_t* y, float inv, bool none) {
    const uint64_t i2 = f2_pack(inv, inv), a = f2_mul(y[0], i2), b = f2_mul(y[1], i2);
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f2_lo(a), f2_hi(a)), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f2_lo(b), f2_hi(b)), __NV_SATFINITE, __NV_E4M3);
    return none ? 0x7f7f7f7fu : lo | (hi << 16);
}
// The codes of a thread's 16 entries under a scale byte (0: none).
template <typename T>
__device__ __forceinline__ void store_codes(uint8_t* block, int l, int left, const uint64_t (&y)[kPer / 2], uint32_t byte) {
    const float inv = __uint_as_float((254u - byte) << 23);
    constexpr int P = Raw<T>::N / 2;  // pairs of a vector
#pragma unroll
    for (int q = 0; q < Raw<T>::V; ++q) {
        if (vec_at<T>(q, l) >= left) continue;
        uint8_t* to = block + vec_at<T>(q, l);
        const uint32_t w = codes4(y + q * P, inv, byte == 0u);
        if (P == 4) *reinterpret_cast<uint2*>(to) = make_uint2(w, codes4(y + q * P + (P == 4 ? 2 : 0), inv, byte == 0u));
        else *reinterpret_cast<uint32_t*>(to) = w;
    }
}
// The bits of the largest |y|, a NaN before everything.
__device__ __forceinline__ uint32_t amax_bits(const uint64_t (&y)[kPer / 2]) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i)
        asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(a) : "f"(a), "f"(f2_lo(y[i])), "f"(f2_hi(y[i])));
    return __float_as_uint(a) & 0x7fffffffu;
}

// A value as a sum of two fp32 numbers. The codes and scales turn on the row's norm, so the last additions of its
// squares, whose roundings do not average out, keep what they lose (in 64 bits they took half of the kernel's time).
struct Two {
    float hi, lo;
};
__device__ __forceinline__ void add(Two& a, float b, float b_lo) {
    const float s = a.hi + b, q = s - a.hi;
    a.lo += ((a.hi - (s - q)) + (b - q)) + b_lo;
    a.hi = s;
}
// The sum of a value over the wpr warps of a row; every thread of the CTA takes part. `red`: 32 floats that this call
// has for itself until two barriers later, zeros where a row has no warp. A row's warps start at a multiple of four
// (or it has fewer than four).
__device__ __forceinline__ Two row_sum(float v, int wpr, float* red) {
    v += __shfl_xor_sync(0xffffffffu, v, 16);
    v += __shfl_xor_sync(0xffffffffu, v, 8);
    if (wpr == 1) {
        Two d{v, 0.0f};
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) add(d, __shfl_xor_sync(0xffffffffu, d.hi, o), __shfl_xor_sync(0xffffffffu, d.lo, o));
        return d;
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, first = warp / wpr * wpr;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    if (wpr == 2) {
        Two d{red[first], 0.0f};
        add(d, red[first + 1], 0.0f);
        return d;
    }
    if (wpr == 3) {
        Two d{red[first] + red[first + 1], 0.0f};
        add(d, red[first + 2], 0.0f);
        return d;
    }
    // (from four warps on a row of the CTA starts at a multiple of four, the CTA's last at its end)
    const float4* r = reinterpret_cast<const float4*>(red + first);
    Two d{0.0f, 0.0f};
    for (int i = 0; i * 4 < wpr; i += 2) {
        const float4 p = r[i], q = (i + 1) * 4 < wpr ? r[i + 1] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        add(d, (p.x + p.y) + (p.z + p.w), 0.0f);
        add(d, (q.x + q.y) + (q.z + q.w), 0.0f);
    }
    return d;
}
// 1 / sqrt(sq * inv + eps), within fp32's rounding of it: the approximation and one step with the whole value.
__device__ __forceinline__ float rsqrt_of(const Two& sq, float inv, float inv_lo, float eps) {
    const float m = sq.hi * inv;
    Two v{m, fmaf(sq.hi, inv, -m) + fmaf(sq.lo, inv, sq.hi * inv_lo)};
    add(v, eps, 0.0f);
    const float r = rsqrtf(v.hi), t = v.hi * r, te = fmaf(v.hi, r, -t);
    const float e = fmaf(-t, r, 1.0f) - (te + v.lo * r) * r;  // 1 - v r^2
    return fmaf(0.5f * r, e, r);
}
__device__ __forceinline__ float squares(const uint64_t (&s)[kPer / 2]) {
    uint64_t t[2] = {0ull, 0ull};
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) t[i & 1] = f2_fma(s[i], s[i], t[i & 1]);
    const uint64_t u = f2_add(t[0], t[1]);
    return f2_lo(u) + f2_hi(u);
}
__device__ __forceinline__ void times(uint64_t (&s)[kPer / 2], float by) {
    const uint64_t b = f2_pack(by, by);
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) s[i] = f2_mul(s[i], b);
}

// Rows on their way while one is reduced, as registers allow.
template <typename T, bool RES, int E>
constexpr int kAheadRows = RES ? (sizeof(T) == 2 ? 1 : 0) : (sizeof(T) == 2 && E == 1 ? 2 : 1);

// E: blocks of a thread, 1 or 2. With two, the instructions that a thread spends on a row whatever its entries (the
// sums, the root, the addresses: a third of 390) serve 32 of them.
template <typename T, bool RES, int E>
__global__ void __launch_bounds__(E == 1 ? 1024 : 512) rmsnorm_fp8_kernel(RmsnormFp8Args a, int wpr) {
    constexpr int A = kAheadRows<T, RES, E>, R = A > 1 ? A : 1;
    __shared__ __align__(16) float red[2][32], red_far[32];
    const int tid = threadIdx.x, warp = tid >> 5, l = tid & 7;
    const int rpc = (blockDim.x >> 5) / wpr;  // rows of a CTA at a time
    const int block = (tid - warp / wpr * wpr * 32) / 8;  // this thread's first block of 128 entries
    const int apart = wpr * 4;                            // blocks from its first to its second
    const int nb = (a.dim + kFp8Block - 1) / kFp8Block;
    const int left = a.dim - block * kFp8Block;  // entries from the first block's start on
    const int rows_step = gridDim.x * rpc;
    if (tid < 32 && tid >= (blockDim.x >> 5)) red[0][tid] = red[1][tid] = red_far[tid] = 0.0f;
    pdl_launch_dependents();
    pdl_wait_prior();
    Raw<T> x[R][E], r[E];
    int row = blockIdx.x * rpc + warp / wpr, next = row;  // (next: the one to load)
    // this thread's first block of row `next` of x; the residual's and the sum's lie at the same distance in every row
    const T* from = static_cast<const T*>(a.x) + static_cast<int64_t>(row) * a.row_stride + block * kFp8Block;
    const int64_t step = static_cast<int64_t>(rows_step) * a.row_stride;
    const int64_t to_residual = static_cast<const char*>(a.residual) - static_cast<const char*>(a.x);
    auto load_row = [&](Raw<T> (&to)[E]) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int n = next < a.rows ? left - e * apart * kFp8Block : 0;
            const T* at = from + e * apart * kFp8Block;
            load16(at, l, n, to[e]);
            if (RES) load16(reinterpret_cast<const T*>(reinterpret_cast<const char*>(at) + to_residual), l, n, r[e]);
        }
        from += step;
        next += rows_step;
    };
    if (A > 0) {
#pragma unroll
        for (int i = 0; i < A; ++i) load_row(x[i]);
    }
    for (int turn = 0, row0 = blockIdx.x * rpc; row0 < a.rows; ++turn, row0 += rows_step, row += rows_step) {  // the CTA's warps together
        if (A == 0) load_row(x[0]);
        const bool live = row < a.rows;
        uint64_t s[E][kPer / 2];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            unpack16(x[0][e], s[e]);
            if (RES) {
                uint64_t t[kPer / 2];
                unpack16(r[e], t);
#pragma unroll
                for (int i = 0; i < kPer / 2; ++i) s[e][i] = f2_add(s[e][i], t[i]);
                T* sum = a.sum ? static_cast<T*>(a.sum) + static_cast<int64_t>(row) * a.row_stride + (block + e * apart) * kFp8Block : nullptr;
                store16(sum, l, live ? left - e * apart * kFp8Block : 0, s[e]);
            }
        }
        if (A > 1) {
#pragma unroll
            for (int e = 0; e < E; ++e) x[0][e] = x[R - 1][e];
        }
        if (A > 0) load_row(x[R - 1]);
        if (a.weight) {  // uniform
            const Two sq = row_sum(E == 1 ? squares(s[0]) : squares(s[0]) + squares(s[E - 1]), wpr, red[turn & 1]);
            float rstd = rsqrt_of(sq, a.inv_dim, a.inv_dim_lo, a.eps);
            // Where the squares, with an eps of their size, leave fp32's range they are summed at 2^-160 and eps is
            // taken there (one that this rounds to 0 is nothing beside them); a row with an infinity or NaN has no norm.
            const bool far = !(sq.hi + a.eps <= 3.0e38f);
            // (the CTA's only row: all its threads alike)
            if (rpc == 1 ? far : wpr == 1 ? __any_sync(0xffffffffu, far) != 0 : __syncthreads_or(far) != 0) {
                constexpr float kDown = 0x1p-80f;
                float part = 0.0f;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    uint64_t low[kPer / 2];
#pragma unroll
                    for (int i = 0; i < kPer / 2; ++i) low[i] = f2_mul(s[e][i], f2_pack(kDown, kDown));
                    part += squares(low);
                }
                const Two lsq = row_sum(part, wpr, red_far);
                if (far) {
#pragma unroll
                    for (int e = 0; e < E; ++e) times(s[e], lsq.hi <= 3.0e38f ? rsqrt_of(lsq, a.inv_dim, a.inv_dim_lo, a.eps * kDown * kDown) : NAN);  // of the row at 2^-80
                    rstd = kDown;
                }
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                Raw<T> w;  // from L1: held in registers it cost the rows on their way more than it saved
                load16(static_cast<const T*>(a.weight) + (block + e * apart) * kFp8Block, l, left - e * apart * kFp8Block, w);
                uint64_t t[kPer / 2];
                unpack16(w, t);
                times(s[e], rstd);
#pragma unroll
                for (int i = 0; i < kPer / 2; ++i) s[e][i] = f2_mul(s[e][i], t[i]);
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int at = block + e * apart, n = left - e * apart * kFp8Block;
            // (entries past the row's end are zeros, or NaN in a row without a norm: not its)
            uint32_t amax = n > 0 ? amax_bits(s[e]) : 0u;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            if (!live) continue;
            const uint32_t byte = scale_byte(amax);
            store_codes<T>(static_cast<uint8_t*>(a.codes) + static_cast<int64_t>(row) * a.dim + at * kFp8Block, l, n, s[e], byte);
            if (l == 0 && at < nb) {
                uint8_t* out = a.scales + static_cast<int64_t>(row) * a.scale_stride;
                out[at] = static_cast<uint8_t>(byte ? byte : 127u);
                if (byte == 0u) raise_status(a.status, kDevNonFinite);
                if (at == nb - 1)  // the row's scales are filled up with zeros
                    for (int b = nb; b < a.scale_stride; ++b) out[b] = 0;
            }
        }
    }
}

// One CTA of 256 threads for each block of 128 x 128: eight lanes a row, four rows a thread.
__global__ void __launch_bounds__(256) fp8_pack_kernel(int N, int K, int scale_stride, const __nv_bfloat16* weight,
                                                       uint8_t* codes, uint8_t* scales) {
    __shared__ uint32_t red[8];
    const int tid = threadIdx.x;
    const int row = blockIdx.y * kFp8Block + tid / 8, col = blockIdx.x * kFp8Block;
    pdl_launch_dependents();
    pdl_wait_prior();
    // thread: lane tid % 8 of the block's row tid / 8 + 32 i
    const int l = tid & 7, left = K - col;
    uint64_t y[4][kPer / 2];
    uint32_t amax = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = row + 32 * i;
        Raw<__nv_bfloat16> r;
        load16(weight + static_cast<size_t>(n) * K + col, l, n < N ? left : 0, r);
        unpack16(r, y[i]);
        amax = max(amax, amax_bits(y[i]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((tid & 31) == 0) red[tid >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, red[i]);
    const uint32_t byte = scale_byte(amax);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = row + 32 * i;
        store_codes<__nv_bfloat16>(codes + static_cast<size_t>(n) * K + col, l, n < N ? left : 0, y[i], byte);
    }
    if (tid == 0) {
        uint8_t* out = scales + static_cast<size_t>(blockIdx.y) * scale_stride;
        out[blockIdx.x] = static_cast<uint8_t>(byte ? byte : 127u);
        if (blockIdx.x == gridDim.x - 1)
            for (int b = gridDim.x; b < scale_stride; ++b) out[b] = 0;
    }
}

}  // namespace

namespace {

template <typename T, bool RES, int E>
cudaError_t launch_rows(const RmsnormFp8Args& a, cudaStream_t stream) {
    // warps of a row: one for 512 (1024) entries, and so many rows that a CTA has kNormThreads
    const int wpr = (a.dim + 32 * kPer * E - 1) / (32 * kPer * E);
    const int rpc = std::max(1, kNormThreads / 32 / wpr), threads = wpr * rpc * 32;
    const int groups = (a.rows + rpc - 1) / rpc;
    auto kernel = rmsnorm_fp8_kernel<T, RES, E>;
    static std::atomic<int> known[33];  // CTAs an SM, by their warps
    int n = known[threads / 32].load(std::memory_order_relaxed);
    if (n == 0) {
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0);
        if (e != cudaSuccess) return e;
        known[threads / 32].store(n = std::max(1, n), std::memory_order_relaxed);
    }
    return launch_pdl(kernel, dim3(static_cast<unsigned>(std::min(groups, 152 * n))), dim3(static_cast<unsigned>(threads)), 0, stream,
                      a, wpr);
}
template <typename T, bool RES>
cudaError_t launch_rows(const RmsnormFp8Args& a, cudaStream_t stream) {
    // Two blocks a thread where there is no residual to load and every SM has rows enough to stay busy with half the
    // threads a row: the instructions bound it then (8001 rows of 8192: fp32 66 -> 55 us, bf16 53 -> 48 us). With a
    // residual the loads do, and fewer threads have fewer on their way (3904 x 5120 bf16: 22.8 -> 26.2 us).
    if constexpr (!RES)
        if (a.dim > 1024 && a.rows > 152 * 4) return launch_rows<T, RES, 2>(a, stream);
    return launch_rows<T, RES, 1>(a, stream);
}

}  // namespace

cudaError_t launch_rmsnorm_fp8(const RmsnormFp8Args& a, int dtype, cudaStream_t stream) {
    if (dtype == 1) return a.residual ? launch_rows<__nv_bfloat16, true>(a, stream) : launch_rows<__nv_bfloat16, false>(a, stream);
    return a.residual ? launch_rows<float, true>(a, stream) : launch_rows<float, false>(a, stream);
}

cudaError_t launch_fp8_pack(int N, int K, int scale_stride, const void* weight, void* codes, uint8_t* scales,
                            cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>((K + kFp8Block - 1) / kFp8Block), static_cast<unsigned>((N + kFp8Block - 1) / kFp8Block));
    return launch_pdl(fp8_pack_kernel, grid, dim3(256), 0, stream, N, K, scale_stride,
                      static_cast<const __nv_bfloat16*>(weight), static_cast<uint8_t*>(codes), scales);
}

}  // namespace eagle
