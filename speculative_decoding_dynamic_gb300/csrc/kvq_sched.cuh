// Work split of the attention over the 8-bit cache, shared by its two kernels
// (k_kvq_decode.cu, k_kvq_attn.cu) and their merge. Not part of the public ABI.
//
// An item is one (sequence, KV head, row block) with all of the sequence's
// keys in steps of `step` keys. The items of all sequences, laid end to end,
// are one line of cost units: `ov` units for an item's start and end, then
// `cost` per step (`cost_last` in a KV head's last item, which may have fewer
// rows). Worker w takes the steps that begin in the units [w chunk, (w+1) chunk),
// whatever the lengths are, so ragged batches, single sequences and long contexts all fill
// the machine; an item that a boundary cuts is finished from its pieces'
// partial results (O, max, sum) by the merge kernel. A worker holds at most
// two pieces of cut items: of the one it continues (slot 2w) and of the one
// it begins (slot 2w + 1). The lengths are device data: every worker derives
// the same line from them by itself.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "eagle_internal.cuh"
#include "quant_ptx.cuh"
#include "quant_ws.h"

namespace eagle {

struct KvqSched {
    const int32_t *prefix_len, *n_tree;  // n_tree may be NULL: T each
    int B, T, max_len;
    int heads, n_items;  // KV heads; items of one
    int step, ov, cost, cost_last, workers, min_chunk;
};

struct KvqSeq {
    int L, n, nkeys, nt;  // nkeys = nt = 0: lengths out of range
    long long len;        // units of a KV head
};

// Units of an item of nt steps.
__device__ __forceinline__ int kvq_units(const KvqSched& s, int nt, bool last) {
    return s.ov + nt * (last ? s.cost_last : s.cost);
}

// SETTLED: the lengths were written before this grid was launched (the
// tensor-core kernel's, behind the split of q, which lets it start only once its
// own wait is over), so that __ldg may read them.
template <bool SETTLED = false>
__device__ __forceinline__ KvqSeq kvq_seq(const KvqSched& s, int b) {
    auto load = [](const int32_t* p) { return SETTLED ? __ldg(p) : ld_prior(p); };
    KvqSeq q;
    q.L = load(&s.prefix_len[b]);
    q.n = s.n_tree ? load(&s.n_tree[b]) : s.T;
    const bool bad = q.L < 0 || q.L > s.max_len - s.T || q.n < 1 || q.n > s.T;
    q.nkeys = bad ? 0 : q.L + q.n;
    q.nt = (q.nkeys + s.step - 1) / s.step;
    q.len = bad ? 0 : (s.n_items - 1) * static_cast<long long>(kvq_units(s, q.nt, false)) + kvq_units(s, q.nt, true);
    return q;
}

// a / b for a >= 0, b > 0: a 64-bit division takes some 150 cycles, and hardly ever is one needed.
__device__ __forceinline__ long long kvq_div(long long a, long long b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

__device__ __forceinline__ long long kvq_chunk(const KvqSched& s, long long total) {
    const long long c = kvq_div(total + s.workers - 1, s.workers);
    return c < s.min_chunk ? s.min_chunk : c;
}

// The sequences' lengths on the line, 32 at a time over a warp's lanes; the
// first kHeld groups are read once, all together, and stay in registers.
struct KvqLens {
    static constexpr int kHeld = 4;
    long long len[kHeld];
    long long total;
    __device__ __forceinline__ long long at(const KvqSched& s, int b) const { return b < s.B ? kvq_seq(s, b).len : 0; }
    __device__ __forceinline__ KvqLens(const KvqSched& s) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) len[i] = at(s, 32 * i + lane);
        long long t = 0;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) t += len[i];
        for (int b = 32 * kHeld + lane; b < s.B; b += 32) t += at(s, b);
        total = static_cast<long long>(warp_sum_u64(static_cast<uint64_t>(t))) * s.heads;
    }
    // The sequence that holds unit pos < total, and the line's length before it (whole warp).
    __device__ __forceinline__ int find(const KvqSched& s, long long pos, long long* base) const {
        const int lane = threadIdx.x & 31;
        long long before = 0;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int l = step(s, len[i], pos, &before, base);
            if (l >= 0) return 32 * i + l;
        }
        for (int b0 = 32 * kHeld; b0 < s.B; b0 += 32) {
            const int l = step(s, at(s, b0 + lane), pos, &before, base);
            if (l >= 0) return b0 + l;
        }
        *base = before;
        return s.B;  // not reached for pos < total
    }

private:
    __device__ __forceinline__ int step(const KvqSched& s, long long own, long long pos, long long* before,
                                        long long* base) const {
        const int lane = threadIdx.x & 31;
        own *= s.heads;
        long long inc = own;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, inc, m);
            if (lane >= m) inc += o;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, *before + inc > pos);
        const int l = hit ? __ffs(hit) - 1 : 31;
        const long long upto = __shfl_sync(0xffffffffu, inc, l), of_l = __shfl_sync(0xffffffffu, own, l);
        if (hit) *base = *before + upto - of_l;
        else *before += upto;
        return hit ? l : -1;
    }
};

// One piece: steps [t0, t1) of item `sub` of sequence b; np: pieces of the
// item if this is its first and it is cut, else 0.
struct KvqPiece {
    int b, sub, L, n, nkeys, nt, t0, t1, np;
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == nt; }
    __device__ __forceinline__ int slot(int worker) const { return 2 * worker + (t0 == 0 ? 1 : 0); }
};

// A worker's pieces in order. init by a whole warp; next by any thread.
struct alignas(16) KvqCursor {
    long long pos, end, base, chunk;
    KvqSeq q;
    int b, worker;
    __device__ __forceinline__ void init(const KvqSched& s, int w) {
        const KvqLens lens(s);
        const long long total = lens.total;
        worker = w;
        chunk = kvq_chunk(s, total);
        pos = min(total, worker * chunk);
        end = min(total, (worker + 1) * chunk);
        base = 0;
        b = 0;
        if (pos < end) {
            b = lens.find(s, pos, &base);
            q = kvq_seq(s, b);
        }
    }
    template <bool SETTLED = false>
    __device__ __forceinline__ bool next(const KvqSched& s, KvqPiece& p) {
        while (pos < end) {
            const long long seq_end = base + q.len * s.heads;
            if (pos >= seq_end) {  // the next sequence with keys (one exists: pos < end <= total)
                base = seq_end;
                do q = kvq_seq<SETTLED>(s, ++b);
                while (q.nt == 0);
                continue;
            }
            const int hk = static_cast<int>(kvq_div(pos - base, q.len));
            const long long head = base + hk * q.len;
            const int full = kvq_units(s, q.nt, false);
            const int i = min(s.n_items - 1, static_cast<int>(kvq_div(pos - head, full)));
            const bool last = i == s.n_items - 1;
            const int cost = last ? s.cost_last : s.cost, units = kvq_units(s, q.nt, last);
            const long long g0 = head + static_cast<long long>(i) * full;
            const int from = static_cast<int>(pos - g0) - s.ov;
            const int to = static_cast<int>(min(static_cast<long long>(units), end - g0)) - s.ov;
            pos = g0 + units;
            p.b = b;
            p.sub = hk * s.n_items + i;
            p.L = q.L;
            p.n = q.n;
            p.nkeys = q.nkeys;
            p.nt = q.nt;
            // the steps that begin in [from, to)
            p.t0 = from <= 0 ? 0 : (from + cost - 1) / cost;
            p.t1 = to <= 0 ? 0 : (to + cost - 1) / cost;
            p.np = 0;  // pieces: up to the worker that has the item's last step
            if (p.t0 == 0 && p.t1 < p.nt)
                p.np = static_cast<int>(kvq_div(g0 + s.ov + static_cast<long long>(p.nt - 1) * cost - worker * chunk, chunk)) + 1;
            if (p.t1 > p.t0) return true;
        }
        return false;
    }
};

// The G*T query rows of a (sequence, KV head): row r <-> tree slot r / G, head hk*G + r % G.
struct KvqRows {
    int G, T, Hq;
    // Row r's slot and its index in the [B*T*Hq] rows of q and out; -1: not a row.
    __device__ __forceinline__ int64_t row(int b, int hk, int r, int* slot) const {
        *slot = r / G;
        if (*slot >= T) return -1;
        return (static_cast<int64_t>(b) * T + *slot) * Hq + static_cast<int64_t>(hk) * G + (r - *slot * G);
    }
};

// Running sum of pieces: (max in the log2 domain, sum, N x 4 columns of O).
template <int N>
struct RowSum {
    float m = -INFINITY, l = 0.0f;
    float4 o[N];
    __device__ __forceinline__ RowSum() {
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    __device__ __forceinline__ void add(float pm, float pl, const float4 (&x)[N]) {
        // a piece in which the row saw nothing: maximum -inf, O 0
        const float M = fmaxf(m, pm);
        const float a = m == -INFINITY ? 0.0f : ex2_approx(m - M), c = pm == -INFINITY ? 0.0f : ex2_approx(pm - M);
        m = M;
        l = l * a + pl * c;
#pragma unroll
        for (int i = 0; i < N; ++i)
            o[i] = make_float4(o[i].x * a + x[i].x * c, o[i].y * a + x[i].y * c, o[i].z * a + x[i].z * c, o[i].w * a + x[i].w * c);
    }
};

// Partial results of cut items: O in units where O / sum is the output, (max
// in the log2 domain, sum) [slot][row][2], and which cut item each worker began:
// (pieces or 0, sequence, item, tree size) [worker]. O is [slot][row][128] for
// the decode kernel; the tensor-core kernel, where a thread owns a row, stores
// [slot][4-column group][row][4] (a row apiece, its stores took 10,000 cycles).
struct KvqPartials {
    float* o;
    float* ml;
    int4* cut;
    int rows;  // rows of a piece
};
__device__ __forceinline__ int4 kvq_cut(const KvqPiece& p) { return make_int4(p.np, p.b, p.sub, p.n); }

struct KvqMergeParams {
    KvqPartials part;
    KvqRows rows;
    int workers, n_items;  // n_items: items of a KV head
    __nv_bfloat16* out;
};
cudaError_t launch_kvq_merge_decode(const KvqMergeParams& p, cudaStream_t stream);

// Zero rows of the sequences whose lengths are out of range (status 3), dealt
// over the workers: `n` threads of a worker, this one the i-th.
template <bool SETTLED = false>
__device__ __forceinline__ void kvq_zero_bad(const KvqSched& s, int Hq, __nv_bfloat16* out, int* status, int worker,
                                             int i, int n) {
    for (int b = worker; b < s.B; b += s.workers) {
        if (kvq_seq<SETTLED>(s, b).nt != 0) continue;
        if (i == 0) raise_status(status, kDevBadIndex);
        uint4* o = reinterpret_cast<uint4*>(out + static_cast<size_t>(b) * s.T * Hq * kKvqHeadDim);
        const int nv = s.T * Hq * kKvqHeadDim / 8;
        for (int e = i; e < nv; e += n) o[e] = make_uint4(0u, 0u, 0u, 0u);
    }
}

// Two e4m3 codes (low and high byte of c) as a pair of fp16: exact.
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t c) {
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(c)));
    return d;
}
// Two floats to a pair of fp16 (a in the low half), nearest even.
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    return d;
}
// A 4-D map of codes: (128 bytes of a head, head, position, sequence), 128-byte swizzle.
inline bool make_map_codes(CUtensorMap* m, const void* base, const KvqDims& kv, int keys) {
    auto fn = tensor_map_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {kKvqHeadDim, static_cast<cuuint64_t>(kv.Hkv), static_cast<cuuint64_t>(kv.max_len),
                                static_cast<cuuint64_t>(kv.B)};
    // a single sequence's stride is never used: any valid one
    const cuuint64_t strides[3] = {kKvqHeadDim, static_cast<cuuint64_t>(kv.pos_stride),
                                   static_cast<cuuint64_t>(kv.B > 1 ? kv.seq_stride : kv.pos_stride)};
    const cuuint32_t box[4] = {kKvqHeadDim, 1, static_cast<cuuint32_t>(keys), 1};
    const cuuint32_t estride[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, estride,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The least reference of V's scales: its reverse is finite (a subnormal scale's need not be).
constexpr float kKvqMinRef = 0x1p-126f;

// Few query rows per KV head: k_kvq_decode.cu.
constexpr int kKvqDecodeRows = 16;
constexpr int kKvqSms = 152;
struct KvqAttnParams {
    KvqSched s;
    KvqPartials part;
    KvqRows rows;
    const float* q_fac;         // tensor-core kernel: factors of the rows of q,
    const KvqCursor* cursors;  // and where its workers start
    int Hq, Hkv, G, W;
    int n_items;    // items of a KV head (pairs of row blocks; 1 in the decode kernel)
    int blk_shift;  // log2 of the positions of a scale block
    int64_t s_seq, s_blk;
    const float *k_scale, *v_scale;  // of this layer
    const __nv_bfloat16* q;
    const uint32_t* mask;  // may be NULL: slot i sees the slots 0..i
    __nv_bfloat16* out;
    int* status;
    float scale_log2;  // log2(e) / sqrt(128)
};
cudaError_t launch_kvq_decode(const KvqDims& kv, const KvqAttnParams& p, const void* kbase, const void* vbase,
                              cudaStream_t stream);
KvqSched kvq_decode_sched(int B, int T, int max_len, int Hkv, int rows);

}  // namespace eagle
