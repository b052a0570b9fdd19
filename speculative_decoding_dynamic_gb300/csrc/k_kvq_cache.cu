// The 8-bit KV cache's writers (sm_103a): eagle_kvq_store and eagle_kvq_compact.
//
// A (sequence, layer, K|V, head) column is cut into blocks of `block`
// positions that share an fp32 scale s; an element is the e4m3 code
// round(x / s). With s a power of two (the smallest with amax <= 448 s) the
// division is exact and so is moving a code to a larger power of two, but for
// values that fall below the format's 2^-6: a block can fill up token by
// token, its scale growing, without losing what earlier tokens had.
//
// Not on the pages: the 16-bit cache's layout and stage 6b in fewer bits.

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "eagle_internal.cuh"
#include "eagle_ws.h"

namespace eagle {
namespace {

constexpr int kD = kKvqHeadDim;
constexpr int kStoreThreads = 256;

// The smallest power of two s >= 2^-126 with amax <= 448 s, amax finite.
// 448 = 1.75 * 2^8: the exponent of amax less 8, one more when its fraction
// is above 1.75.
__device__ __forceinline__ float block_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // biased by 127
    return __uint_as_float(static_cast<uint32_t>(max(e, 1)) << 23);
}

__device__ __forceinline__ bool pow2(float s) { return (__float_as_uint(s) & 0x7fffffu) == 0u; }

// Two values to two e4m3 codes (the first in the low byte), nearest even, saturating.
__device__ __forceinline__ uint32_t codes2(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float2 values2(uint32_t c2) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c2), __NV_E4M3);
    return __half22float2(__half2(h));
}

// Four codes moved from scale s_old to s_new: code * (s_old / s_new).
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
    const float2 lo = values2(w & 0xffffu), hi = values2(w >> 16);
    return codes2(lo.x * ratio, lo.y * ratio) | (codes2(hi.x * ratio, hi.y * ratio) << 16);
}

// One group of 2 * BLK threads per (sequence, block, K|V, head): every thread
// holds eight 16-byte pieces (64 elements) of the block's rows in registers,
// so the tokens are read once: amax, scale, codes. 16 threads read one
// 256-byte row and write its 128 bytes of codes; a CTA of 256 threads takes
// 256 / (2 BLK) neighbouring heads.
//
// Bound by HBM: two bytes read and one written per element. Holding the block
// in registers instead of reading it a second time for the codes is why the
// group grows with the block.
template <int BLK>
__global__ void __launch_bounds__(kStoreThreads) kvq_store_kernel(
    KvqDims kv, int layer, int T, int nhg, const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
    int64_t row_stride, const int32_t* __restrict__ row_start, const int32_t* __restrict__ start,
    const int32_t* __restrict__ count, unsigned char* __restrict__ codes, float* __restrict__ scales, int* status) {
    constexpr int GT = 2 * BLK;                 // threads of a group
    constexpr int GROUPS = kStoreThreads / GT;  // groups (heads) per CTA
    constexpr int ROWS = BLK / 8;               // rows per pass
    __shared__ uint32_t wmax[kStoreThreads / 32];
    const int b = blockIdx.z, which = blockIdx.y;
    const int tid = threadIdx.x;
    const int h = (blockIdx.x % nhg) * GROUPS + tid / GT;
    const int gt = tid % GT;
    pdl_launch_dependents();
    pdl_wait_prior();
    const int p0 = start[b];
    const int n = count ? count[b] : T;
    const int64_t r0 = row_start ? row_start[b] : static_cast<int64_t>(b) * T;
    // n > 0 first: the comparisons on p0 cannot overflow after the check
    if (n < 0 || n > T || p0 < 0 || p0 > kv.max_len - n || r0 < 0) {
        if (tid == 0 && blockIdx.x == 0 && which == 0) raise_status(status, kDevBadIndex);
        return;
    }
    const int blk = p0 / BLK + static_cast<int>(blockIdx.x) / nhg;
    const int lo = blk * BLK;  // first position of the block
    if (n == 0 || lo >= p0 + n) return;  // uniform over the CTA
    const bool live = h < kv.Hkv;
    const __nv_bfloat16* src = which ? v : k;
    unsigned char* dst = codes + b * kv.seq_stride + layer * kv.layer_stride + which * kv.kv_stride +
                         static_cast<int64_t>(h) * kD;
    float* sp = scales + b * kv.s_seq + layer * kv.s_layer + which * kv.s_kv + blk * kv.s_blk + h;
    const bool merge = lo < p0;  // the block holds earlier positions
    const float s_old = live && merge ? *sp : 0.0f;
    const int col = gt % 16;
    uint4 x[8];
    uint32_t mx = 0u;  // packed largest |x| of two bf16 columns (a NaN is above infinity)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int pos = lo + i * ROWS + gt / 16;
        const bool in = live && pos >= p0 && pos < p0 + n;
        x[i] = in ? __ldcs(reinterpret_cast<const uint4*>(src + (r0 + (pos - p0)) * row_stride +
                                                          static_cast<int64_t>(h) * kD) + col)
                  : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t m01 = __vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu);
        const uint32_t m23 = __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu);
        mx = __vmaxu2(mx, __vmaxu2(m01, m23));
    }
    uint32_t am = max(mx & 0xffffu, mx >> 16);
    am = __reduce_max_sync(0xffffffffu, am);
    if (GT > 32) {
        if ((tid & 31) == 0) wmax[tid >> 5] = am;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < GT / 32; ++i) am = max(am, wmax[tid / GT * (GT / 32) + i]);
    }
    if (!live) return;
    if (am >= 0x7f80u) {  // NaN or infinity among the new elements
        if (gt == 0) raise_status(status, kDevNonFinite);
        am = 0x7f7fu;
    }
    float s = block_scale(__uint_as_float(am << 16));
    if (merge) s = fmaxf(s, s_old);
    if (gt == 0) *sp = s;
    const bool exact = pow2(s);
    const float inv = 1.0f / s;  // exact for a power of two (2^-126 .. 2^120)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int pos = lo + i * ROWS + gt / 16;
        uint2* out = reinterpret_cast<uint2*>(dst + pos * kv.pos_stride) + col;
        if (pos >= p0 && pos < p0 + n) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            uint32_t c[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float a = __uint_as_float(w[e] << 16), d = __uint_as_float(w[e] & 0xffff0000u);
                c[e] = exact ? codes2(a * inv, d * inv) : codes2(__fdiv_rn(a, s), __fdiv_rn(d, s));
            }
            *out = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
        } else if (merge && pos < p0 && s > s_old) {  // earlier tokens of the block, at the grown scale
            const float ratio = __fdiv_rn(s_old, s);
            const uint2 w = *out;
            *out = make_uint2(rescale4(w.x, ratio), rescale4(w.y, ratio));
        }
    }
}

constexpr int kMoveWarps = 4;
constexpr int kMaxAccept = kMaxDepth;  // a_b <= D <= 16 <= block: destinations span two blocks at most

// One warp per (sequence, layer, K|V, head): a row of codes is 128 bytes, four
// per lane. Every source row is in registers before the first store, and a
// lane rewrites only bytes that it alone reads, so no barrier is needed. A
// chain of dependent small loads (lengths, slots, rows and scales) and its
// latency are the whole cost; the slots and the scales of all rows are loaded
// by the lanes at once.
__global__ void __launch_bounds__(kMoveWarps * 32) kvq_compact_kernel(
    KvqDims kv, unsigned char* __restrict__ codes, float* __restrict__ scales, const int32_t* __restrict__ prefix_len,
    const int32_t* __restrict__ accept_len, const int32_t* __restrict__ slots, int slots_stride,
    int32_t* __restrict__ new_len, int* status) {
    const int b = blockIdx.z;
    const int layer = blockIdx.y >> 1, which = blockIdx.y & 1;
    const int lane = threadIdx.x & 31;
    const int h = blockIdx.x * kMoveWarps + (threadIdx.x >> 5);
    pdl_launch_dependents();
    pdl_wait_prior();
    const int L = prefix_len[b], a = accept_len[b];
    bool ok = a >= 0 && a <= kMaxAccept && a < slots_stride && L >= 0 && L < kv.max_len - a;
    // lane j holds row j: its slot, whether it moves
    int sj = lane;
    if (ok && lane >= 1 && lane <= a) sj = slots[static_cast<int64_t>(b) * slots_stride + lane];
    ok = ok && !__any_sync(0xffffffffu, lane >= 1 && lane <= a && (sj < lane || sj >= kv.max_len - L));
    const bool first = blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0;
    if (!ok) {
        if (first) raise_status(status, kDevBadIndex);
        return;
    }
    if (first) new_len[b] = L + a + 1;
    if (h >= kv.Hkv) return;
    const unsigned moving = __ballot_sync(0xffffffffu, sj > lane);
    if (moving == 0u) return;
    unsigned char* col = codes + b * kv.seq_stride + layer * kv.layer_stride + which * kv.kv_stride +
                         static_cast<int64_t>(h) * kD + lane * 4;
    float* sc = scales + b * kv.s_seq + layer * kv.s_layer + which * kv.s_kv + h;
    uint32_t row[kMaxAccept];
#pragma unroll
    for (int j = 1; j <= kMaxAccept; ++j) {
        const int s = __shfl_sync(0xffffffffu, sj, j);
        if (j <= a && s > j) row[j - 1] = *reinterpret_cast<const uint32_t*>(col + (L + s) * kv.pos_stride);
    }
    const bool mine = sj > lane;
    const float s_src = mine ? sc[static_cast<int64_t>((L + sj) / kv.block) * kv.s_blk] : 0.0f;
    const int blk0 = (L + 1) / kv.block;
    const int blk_of = (L + lane) / kv.block;  // block of this lane's destination
    float s_new = 0.0f;  // the new scale of this lane's destination block
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int blk = blk0 + i;
        const unsigned into = __ballot_sync(0xffffffffu, mine && blk_of == blk);
        if (into == 0u) continue;
        const float had = sc[static_cast<int64_t>(blk) * kv.s_blk];
        float s = mine && blk_of == blk ? s_src : 0.0f;
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) s = fmaxf(s, __shfl_xor_sync(0xffffffffu, s, m));
        s = fmaxf(s, had);
        if (blk_of == blk) s_new = s;
        if (s > had) {  // the block's scale grows: its other rows move to it
            const float ratio = __fdiv_rn(had, s);
            const int hi = min((blk + 1) * kv.block, L + a + 1);
            for (int pos = blk * kv.block; pos < hi; ++pos) {
                uint32_t* w = reinterpret_cast<uint32_t*>(col + pos * kv.pos_stride);
                const int j = pos - L;
                if (j < 1 || !((moving >> j) & 1u)) *w = rescale4(*w, ratio);
            }
            __syncwarp();
            if (lane == 0) sc[static_cast<int64_t>(blk) * kv.s_blk] = s;
        }
    }
    const float ratio = mine ? __fdiv_rn(s_src, s_new) : 1.0f;
#pragma unroll
    for (int j = 1; j <= kMaxAccept; ++j) {
        const float r = __shfl_sync(0xffffffffu, ratio, j);
        if ((moving >> j) & 1u)
            *reinterpret_cast<uint32_t*>(col + (L + j) * kv.pos_stride) = r == 1.0f ? row[j - 1] : rescale4(row[j - 1], r);
    }
}

template <int BLK>
cudaError_t store(const KvqDims& kv, int layer, int T, const void* k, const void* v, int64_t row_stride,
                  const int32_t* row_start, const int32_t* start, const int32_t* count, void* codes, float* scales,
                  int* status, cudaStream_t stream) {
    constexpr int GROUPS = kStoreThreads / (2 * BLK);
    const int nhg = (kv.Hkv + GROUPS - 1) / GROUPS;
    const long nblk = std::min<long>((static_cast<long>(std::min(T, kv.max_len)) + BLK - 2) / BLK + 1,
                                     (kv.max_len + BLK - 1L) / BLK);  // blocks a sequence's tokens can touch
    if (nblk * nhg > 0x7fffffffL) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(nblk * nhg), 2, kv.B);
    return launch_pdl(kvq_store_kernel<BLK>, grid, dim3(kStoreThreads), 0, stream, kv, layer, T, nhg,
                      static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), row_stride, row_start,
                      start, count, static_cast<unsigned char*>(codes), scales, status);
}

}  // namespace

cudaError_t launch_kvq_store(const KvqDims& kv, int layer, int T, const void* k, const void* v, int64_t row_stride,
                             const int32_t* row_start, const int32_t* start, const int32_t* count, void* codes,
                             float* scales, int* status, cudaStream_t stream) {
    auto fn = kv.block == 16 ? store<16> : kv.block == 32 ? store<32> : kv.block == 64 ? store<64> : store<128>;
    return fn(kv, layer, T, k, v, row_stride, row_start, start, count, codes, scales, status, stream);
}

cudaError_t launch_kvq_compact(const KvqDims& kv, void* codes, float* scales, const int32_t* prefix_len,
                               const int32_t* accept_len, const int32_t* slots, int slots_stride, int32_t* new_len,
                               int* status, cudaStream_t stream) {
    const dim3 grid((kv.Hkv + kMoveWarps - 1) / kMoveWarps, kv.layers * 2, kv.B);
    return launch_pdl(kvq_compact_kernel, grid, dim3(kMoveWarps * 32), 0, stream, kv,
                      static_cast<unsigned char*>(codes), scales, prefix_len, accept_len, slots, slots_stride, new_len,
                      status);
}

}  // namespace eagle
