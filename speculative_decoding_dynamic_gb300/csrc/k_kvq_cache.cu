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
#include "quant_ws.h"

namespace eagle {
namespace {

constexpr int kD = kKvqHeadDim;
constexpr int kStoreThreads = 256;

// The kernels' inputs are not __restrict__: a const __restrict__ input may be
// read like one by __ldg, which wants data that nothing writes while the grid
// runs, and under programmatic launch the kernel that writes it may still run.

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
// group grows with the block. Measured: 20,000 prompt tokens of 40 heads (461 MB)
// 71.4 us, 6.5 TB/s; 64 trees of 61 slots of 8 heads (24 MB) 5.5 us in a captured graph.
template <int BLK>
__global__ void __launch_bounds__(kStoreThreads) kvq_store_kernel(
    KvqDims kv, int layer, int T, int nhg, const __nv_bfloat16* k, const __nv_bfloat16* v,
    int64_t row_stride, const int32_t* row_start, const int32_t* start,
    const int32_t* count, unsigned char* __restrict__ codes, float* __restrict__ scales, int* status) {
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
    // this thread's 16-byte column of rows gt / 16, gt / 16 + ROWS, ..
    const int pos0 = lo + gt / 16, col = gt % 16;
    const bool full = lo >= p0 && lo + BLK <= p0 + n;  // every position of the block is new
    const uint4* in = reinterpret_cast<const uint4*>(src + (r0 + (pos0 - p0)) * row_stride + static_cast<int64_t>(h) * kD) + col;
    const int64_t in_step = row_stride * ROWS / 8;
    uint4 x[8];
    uint32_t mx = 0u;  // packed largest |x| of two bf16 columns (a NaN is above infinity)
    if (full && live) {
#pragma unroll
        for (int i = 0; i < 8; ++i, in += in_step) x[i] = __ldcs(in);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i, in += in_step)
            x[i] = live && static_cast<unsigned>(pos0 + i * ROWS - p0) < static_cast<unsigned>(n) ? __ldcs(in)
                                                                                                   : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
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
    const int64_t out_step = kv.pos_stride * ROWS / 8;
    uint2* out = reinterpret_cast<uint2*>(dst + pos0 * kv.pos_stride) + col;
    if (merge && s > s_old) {  // earlier tokens of the block, at the grown scale
        const float ratio = __fdiv_rn(s_old, s);
        uint2* w = out;
        for (int i = 0; i < 8 && pos0 + i * ROWS < p0; ++i, w += out_step) {
            const uint2 u = *w;
            *w = make_uint2(rescale4(u.x, ratio), rescale4(u.y, ratio));
        }
    }
    if (!pow2(s)) {  // an old scale from elsewhere: x / s as a division
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            // x[i] by a select: an index that varies would put the array in local memory
            uint4 u = x[0];
#pragma unroll
            for (int e = 1; e < 8; ++e)
                if (i == e) u = x[e];
            if (static_cast<unsigned>(pos0 + i * ROWS - p0) >= static_cast<unsigned>(n)) continue;
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
            uint32_t c[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                c[e] = codes2(__fdiv_rn(__uint_as_float(w[e] << 16), s), __fdiv_rn(__uint_as_float(w[e] & 0xffff0000u), s));
            out[i * out_step] = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
        }
        return;
    }
    const float inv = 1.0f / s;  // exact for a power of two (2^-126 .. 2^120)
    const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll
    for (int i = 0; i < 8; ++i, out += out_step) {
        if (!full && static_cast<unsigned>(pos0 + i * ROWS - p0) >= static_cast<unsigned>(n)) continue;
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint64_t q = f2_mul(f2_pack(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u)), inv2);
            c[e] = codes2(f2_lo(q), f2_hi(q));
        }
        *out = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    }
}

constexpr int kMoveWarps = 2;
constexpr int kMoveHeads = 4;          // heads of a warp, eight lanes each
constexpr int kMaxAccept = kMaxDepth;  // a_b <= D <= 16 <= block: destinations span two blocks at most

// Sixteen codes moved to another scale.
__device__ __forceinline__ uint4 rescale16(const uint4& u, float ratio) {
    return make_uint4(rescale4(u.x, ratio), rescale4(u.y, ratio), rescale4(u.z, ratio), rescale4(u.w, ratio));
}

// One warp per (sequence, layer, K|V, four heads): a lane holds 16 bytes of a
// row and every source row is in registers before the first store; a lane
// rewrites only bytes that it alone reads, so no barrier is needed. The cost
// is a chain of small loads (lengths and slots, then rows and scales) and
// the number of warps that go through it: four heads per warp bring a batch
// of 64 with 32 layers into one wave (one head per warp: 16.8 us; four: 9.1, and
// 2.8 us for one sequence, in a captured graph on a cache that it has compacted before;
// 27 and 5 us on a fresh one, where the scales of destination blocks grow).
__global__ void __launch_bounds__(kMoveWarps * 32) kvq_compact_kernel(
    KvqDims kv, unsigned char* __restrict__ codes, float* __restrict__ scales, const int32_t* prefix_len,
    const int32_t* accept_len, const int32_t* slots, int slots_stride,
    int32_t* __restrict__ new_len, int* status) {
    const int b = blockIdx.z;
    const int layer = blockIdx.y >> 1, which = blockIdx.y & 1;
    const int lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait_prior();
    const int L = prefix_len[b], a = accept_len[b];
    // lane j holds row j: its slot, whether it moves
    int sj = lane;
    if (lane >= 1 && lane < min(slots_stride, kMaxAccept + 1)) sj = slots[static_cast<int64_t>(b) * slots_stride + lane];
    if (lane > a) sj = lane;
    bool ok = a >= 0 && a <= kMaxAccept && a < slots_stride && L >= 0 && L < kv.max_len - a;
    ok = ok && !__any_sync(0xffffffffu, lane >= 1 && lane <= a && (sj < lane || sj >= kv.max_len - L));
    const bool first = blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0;
    if (!ok) {
        if (first) raise_status(status, kDevBadIndex);
        return;
    }
    if (first) new_len[b] = L + a + 1;
    const unsigned moving = __ballot_sync(0xffffffffu, sj > lane);
    if (moving == 0u) return;
    const int h = (blockIdx.x * kMoveWarps + (threadIdx.x >> 5)) * kMoveHeads + (lane >> 3);
    const bool live = h < kv.Hkv;
    const int q = lane & 7;
    unsigned char* col = codes + b * kv.seq_stride + layer * kv.layer_stride + which * kv.kv_stride +
                         static_cast<int64_t>(h) * kD + q * 16;
    float* sc = scales + b * kv.s_seq + layer * kv.s_layer + which * kv.s_kv + h;
    uint4 row[kMaxAccept];
#pragma unroll
    for (int j = 1; j <= kMaxAccept; ++j) {
        const int s = __shfl_sync(0xffffffffu, sj, j);
        if (live && s > j) row[j - 1] = *reinterpret_cast<const uint4*>(col + (L + s) * kv.pos_stride);
    }
    // lane q of a head holds the scales of rows q + 1 and q + 9
    const int blk0 = (L + 1) / kv.block;
    float had[2] = {0.0f, 0.0f}, s_src[2], s_new[2] = {0.0f, 0.0f};
    int blk_of[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int j = q + 1 + 8 * e;
        const int s = __shfl_sync(0xffffffffu, sj, j);
        const bool moves = live && ((moving >> j) & 1u);
        s_src[e] = moves ? sc[static_cast<int64_t>((L + s) / kv.block) * kv.s_blk] : 0.0f;
        blk_of[e] = moves ? (L + j) / kv.block - blk0 : -1;
        if (live && L + 1 + e * (kv.block - (L + 1) % kv.block) <= L + a)  // block blk0 + e holds a destination
            had[e] = sc[static_cast<int64_t>(blk0 + e) * kv.s_blk];
    }
    float grown[2];  // the old scale over the new of the (up to two) destination blocks
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float s = fmaxf(blk_of[0] == i ? s_src[0] : 0.0f, blk_of[1] == i ? s_src[1] : 0.0f);
#pragma unroll
        for (int m = 4; m > 0; m >>= 1) s = fmaxf(s, __shfl_xor_sync(0xffffffffu, s, m));
        s = fmaxf(s, had[i]);
        grown[i] = s > had[i] ? __fdiv_rn(had[i], s) : 1.0f;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (blk_of[e] == i) s_new[e] = s;
        if (q == 0 && s > had[i]) sc[static_cast<int64_t>(blk0 + i) * kv.s_blk] = s;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (!live || grown[i] == 1.0f) continue;  // uniform over a head's lanes
        const int hi = min((blk0 + i + 1) * kv.block, L + a + 1);
        // the block's other rows move to its grown scale, four read at once (one after the other, each
        // waited for the one before: 44 us for 64 cold sequences of 8B against 30; eight: 32)
        for (int pos = (blk0 + i) * kv.block; pos < hi; pos += 4) {
            uint4 w[4];
            bool stays[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = pos + e - L;
                stays[e] = pos + e < hi && !(j >= 1 && ((moving >> j) & 1u));
                if (stays[e]) w[e] = *reinterpret_cast<const uint4*>(col + (pos + e) * kv.pos_stride);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (stays[e]) *reinterpret_cast<uint4*>(col + (pos + e) * kv.pos_stride) = rescale16(w[e], grown[i]);
        }
    }
    const float ratio[2] = {blk_of[0] >= 0 ? __fdiv_rn(s_src[0], s_new[0]) : 1.0f,
                            blk_of[1] >= 0 ? __fdiv_rn(s_src[1], s_new[1]) : 1.0f};
#pragma unroll
    for (int j = 1; j <= kMaxAccept; ++j) {
        const float r = __shfl_sync(0xffffffffu, ratio[(j - 1) >> 3], (lane & 24) + ((j - 1) & 7));
        if (live && ((moving >> j) & 1u))
            *reinterpret_cast<uint4*>(col + (L + j) * kv.pos_stride) = r == 1.0f ? row[j - 1] : rescale16(row[j - 1], r);
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
    constexpr int per_cta = kMoveWarps * kMoveHeads;
    const dim3 grid((kv.Hkv + per_cta - 1) / per_cta, kv.layers * 2, kv.B);
    return launch_pdl(kvq_compact_kernel, grid, dim3(kMoveWarps * 32), 0, stream, kv,
                      static_cast<unsigned char*>(codes), scales, prefix_len, accept_len, slots, slots_stride, new_len,
                      status);
}

}  // namespace eagle
