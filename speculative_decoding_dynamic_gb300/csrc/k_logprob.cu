// Log-probabilities of given tokens with rank, entropy and top alternatives
// (sm_103a): eagle_token_logprobs. Not on the pages; the rows are the target
// rows of stage 6.
//
// With c = log2(e) / T, the row's maximum M and y = (x - M) c:
//   S = sum 2^y, E = sum y 2^y
//   ln p[t] = (x_t - M) / T - ln S,  entropy = ln S - ln2 E / S
// M is a reference here, at most 4 / c below the row's maximum: S and E are
// kept together in one pass, like an online softmax, and when the reference
// rises by d / c, S <- 2^-d S and E <- 2^-d (E - d S). It rises only when
// an entry is more than 4 / c above it, so hardly ever after a thread's first
// group (at every new maximum some lane of a warp had one in most groups). The
// difference is taken before the product (one packed addition more than a
// multiply-add of the scaled maximum) so that it is exact next to logits of any
// size. The rank counts entries above the token's logit, read before the pass.
// y is kept above -2^100 (2^y is 0 there, and y 2^y must not be -inf * 0), and
// so is the reference.
//
// Bound by HBM: a row is read once, 16 bytes per lane and load, four loads in
// flight per thread, and other CTAs' loads (six per SM for fp32 rows, four for
// bf16 ones, whose unpacking needs the registers) behind a CTA's arithmetic and
// tail. About six instructions per element beside the one exponential
// (packed fp32 pairs for the multiply-adds and sums, packed bf16 for maxima and
// compares; the compare is skipped for groups whose maximum is below the
// token's logit). Measured: 4096 fp32 rows of 32000 (524 MB) 99 us, 79% of HBM;
// some 250 bf16 rows of 128256 (65 MB) 22.2 us, a wave of CTAs. A row is split over a cluster of
// 1..8 CTAs when there are few rows. The alternatives need no second pass
// over the row: the k-th largest of the threads' maxima bounds the k-th
// largest entry from below, and only the groups (four vectors of a thread)
// whose maximum reaches it are read again, from L2.

#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "eagle_internal.cuh"
#include "quant_ptx.cuh"
#include "quant_ws.h"

namespace eagle {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kVecs = 4;                             // 16-byte vectors of a group
constexpr int kChunkBytes = kThreads * kVecs * 16;   // 16 KB
constexpr int kKeys = 512;                           // candidate keys held at once
constexpr int kGroups = 512;                         // groups read again at once
constexpr float kFloor = -0x1p100f;  // a value of both types
constexpr float kLog2e = 1.4426950408889634f;

struct Part {  // one CTA's share of a row
    float m, s, e;
    int above;
};
struct Shared {
    alignas(16) uint32_t wtop[kWarps * kMaxTopK];
    unsigned long long keys[kKeys];
    unsigned long long red[kWarps];
    uint64_t ctop[kMaxTopK];
    Part wpart[kWarps];
    float wmax[kWarps];
    int nkeys, ngroups;
    uint32_t tau;
    uint32_t groups[kGroups];  // (chunk, thread) of the groups that reach tau
    // filled by every CTA of the cluster in the leader's copy
    uint64_t rtop[kMaxChunks * kMaxTopK];
    Part rpart[kMaxChunks];
    float rmax[kMaxChunks];
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ __nv_bfloat162 bf2(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }

template <int DT>
__device__ __forceinline__ float vec_max(const uint4& u) {
    if (DT == 1) {
        const __nv_bfloat162 m = __hmax2(__hmax2(bf2(u.x), bf2(u.y)), __hmax2(bf2(u.z), bf2(u.w)));
        return fmaxf(__low2float(m), __high2float(m));
    }
    return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
}
template <int DT>
__device__ __forceinline__ float element(const uint4& u, int e) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if (DT == 1) return __uint_as_float((e & 1) ? (w[e >> 1] & 0xffff0000u) : (w[e >> 1] << 16));
    return __uint_as_float(w[e]);
}
template <int DT>
__device__ __forceinline__ uint4 neg_inf() {
    const uint32_t w = DT == 1 ? 0xff80ff80u : 0xff800000u;
    return make_uint4(w, w, w, w);
}

// Entries of N vectors above x.
template <int DT, int N>
__device__ __forceinline__ int count_above(const uint4* u, float x) {
    if (DT == 1) {
        // x is a bf16 value, or the fp32 value below one: rounding it down to bf16 keeps the order of bf16 entries
        const __nv_bfloat16 h = __float2bfloat16_rd(x);
        const __nv_bfloat162 t = __halves2bfloat162(h, h);
        __nv_bfloat162 n[2];  // at most 8 N a half: exact
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const __nv_bfloat162 a = __hadd2(__hgt2(bf2(u[q].x), t), __hgt2(bf2(u[q].y), t));
            const __nv_bfloat162 b = __hadd2(__hgt2(bf2(u[q].z), t), __hgt2(bf2(u[q].w), t));
            n[0] = q ? __hadd2(n[0], a) : a;
            n[1] = q ? __hadd2(n[1], b) : b;
        }
        const __nv_bfloat162 all = __hadd2(n[0], n[1]);
        return static_cast<int>(__low2float(all) + __high2float(all));
    }
    // the signs of x - entry, two per packed instruction (of equal infinities NaN, whose sign is clear)
    x += 0.0f;  // of -0, 0 - entry would be negative for an entry of 0
    const uint64_t minus = f2_pack(-1.0f, -1.0f), x2 = f2_pack(x, x);
    uint32_t n = 0u;
#pragma unroll
    for (int q = 0; q < N; ++q) {
        const uint64_t a = f2_fma((static_cast<uint64_t>(u[q].y) << 32) | u[q].x, minus, x2);
        const uint64_t b = f2_fma((static_cast<uint64_t>(u[q].w) << 32) | u[q].z, minus, x2);
        n += __float_as_uint(f2_lo(a)) >> 31;
        n += __float_as_uint(f2_hi(a)) >> 31;
        n += __float_as_uint(f2_lo(b)) >> 31;
        n += __float_as_uint(f2_hi(b)) >> 31;
    }
    return static_cast<int>(n);
}

// a <- a and b over the larger maximum.
__device__ __forceinline__ void join(Part& a, const Part& b, float c) {
    const float M = fmaxf(a.m, b.m);
    const float da = a.m == -INFINITY ? 0.0f : (a.m - M) * c, db = b.m == -INFINITY ? 0.0f : (b.m - M) * c;
    const float fa = a.m == -INFINITY ? 0.0f : ex2_approx(da), fb = b.m == -INFINITY ? 0.0f : ex2_approx(db);
    // a factor of 0 comes with a difference that may be infinite
    a.e = (fa > 0.0f ? fa * fmaf(da, a.s, a.e) : 0.0f * a.s) + (fb > 0.0f ? fb * fmaf(db, b.s, b.e) : 0.0f * b.s);
    a.s = fa * a.s + fb * b.s;
    a.m = M;
    a.above += b.above;
}

// The parts of 2^STEPS neighbouring lanes joined in all of them: their common reference, then plain sums.
template <int STEPS>
__device__ __forceinline__ void join_lanes(Part& a, float c) {
    float M = a.m;
#pragma unroll
    for (int o = 1; o < 1 << STEPS; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float d = a.m == -INFINITY ? 0.0f : (a.m - M) * c, f = a.m == -INFINITY ? 0.0f : ex2_approx(d);
    a.e = f > 0.0f ? f * fmaf(d, a.s, a.e) : f * a.s;  // a factor of 0 comes with a difference that may be infinite
    a.s = f * a.s;
    a.m = M;
#pragma unroll
    for (int o = 1; o < 1 << STEPS; o <<= 1) {
        a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
        a.e += __shfl_xor_sync(0xffffffffu, a.e, o);
        a.above += __shfl_xor_sync(0xffffffffu, a.above, o);
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads, DT == 1 ? 4 : 6) token_logprobs_kernel(LogprobArgs a, int cpr, int seg, float c) {
    extern __shared__ __align__(16) unsigned char gmax_raw[];  // [chunk][thread] group maxima (ordered bits)
    __shared__ Shared sm;
    constexpr int ES = DT == 1 ? 2 : 4;
    constexpr int EPV = 16 / ES;
    constexpr int CE = kChunkBytes / ES;  // elements of a chunk
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int entry = blockIdx.x / cpr, rank = blockIdx.x % cpr;  // a cluster is cpr neighbouring CTAs
    const int k = a.n_alt;
    pdl_launch_dependents();
    pdl_wait_prior();
    const int b = entry / a.per_seq, j = entry - b * a.per_seq;
    const int slot = a.slots ? a.slots[entry] : j;
    const int tok = a.tokens[entry];
    if (slot < 0 || tok < 0 || slot >= a.rows_per_seq || tok >= a.V) {  // uniform over the cluster
        if (rank == 0) {
            if (tid == 0) {
                if (slot >= a.rows_per_seq || tok >= a.V) raise_status(a.status, kDevBadIndex);
                a.logprob[entry] = NAN;
                if (a.entropy) a.entropy[entry] = NAN;
                if (a.rank) a.rank[entry] = -1;
            }
            if (tid < k) {
                a.alt_ids[static_cast<size_t>(entry) * k + tid] = -1;
                a.alt_logprobs[static_cast<size_t>(entry) * k + tid] = NAN;
            }
        }
        return;
    }
    if (cpr > 1) cluster_started_arrive();
    const char* row = static_cast<const char*>(a.logits) +
                      (static_cast<size_t>(b) * a.rows_per_seq + slot) * static_cast<size_t>(a.V) * ES;
    const int first = rank * seg;                       // this CTA's elements [first, first + n)
    const int n = max(0, min(seg, a.V - first));
    const int nch = (n + CE - 1) / CE;
    const uint4* vec = reinterpret_cast<const uint4*>(row + static_cast<size_t>(first) * ES);
    const int nvec = n / EPV;
    const float xt = DT == 1 ? __uint_as_float(static_cast<uint32_t>(ld_prior(reinterpret_cast<const unsigned short*>(row) + tok)) << 16)
                             : ld_prior(reinterpret_cast<const float*>(row) + tok);
    // x >= xt as x > xt_below, the next value down (both zeros are one value)
    const float xt_below = xt == 0.0f ? __uint_as_float(0x80000001u) : o2f(f2o(xt) - 1u);
    if (tid == 0) {
        sm.nkeys = sm.ngroups = 0;
        sm.tau = 0u;
    }
    if (tid < kMaxTopK) sm.ctop[tid] = 0ull;

    // ---- the pass ----
    Part my{-INFINITY, 0.0f, 0.0f, 0};
    float top = -INFINITY;  // this thread's largest element
    const uint64_t c2 = f2_pack(c, c);
    const int tokv = tok / EPV - first / EPV;  // the token's vector in this CTA's numbering (first is a multiple of EPV)
    auto load = [&](int ch, uint4 (&u)[kVecs]) {
        if (ch >= nch) return;
        const uint4* in = vec + ch * kVecs * kThreads + tid;
        if ((ch + 1) * kVecs * kThreads <= nvec) {
#pragma unroll
            for (int q = 0; q < kVecs; ++q) u[q] = ld_prior(in + q * kThreads);
        } else {
            const int v0 = ch * kVecs * kThreads + tid;
#pragma unroll
            for (int q = 0; q < kVecs; ++q) u[q] = v0 + q * kThreads < nvec ? ld_prior(in + q * kThreads) : neg_inf<DT>();
        }
    };
    auto group = [&](int ch, const uint4 (&u)[kVecs]) {
        if (ch >= nch) return;
        const int v0 = ch * kVecs * kThreads + tid;
        const float gm = fmaxf(fmaxf(vec_max<DT>(u[0]), vec_max<DT>(u[1])), fmaxf(vec_max<DT>(u[2]), vec_max<DT>(u[3])));
        const bool any = v0 < nvec;
        top = fmaxf(top, gm);
        if (k > 0) {  // bf16 values are decided by the top half of their ordered bits
            if (DT == 1) reinterpret_cast<uint16_t*>(gmax_raw)[ch * kThreads + tid] = any ? f2o(gm) >> 16 : 0;
            else reinterpret_cast<uint32_t*>(gmax_raw)[ch * kThreads + tid] = any ? f2o(gm) : 0u;
        }
        if (!any) return;
        if (gm >= xt && xt > -INFINITY && (v0 > tokv || v0 + (kVecs - 1) * kThreads < tokv)) {
            // vectors before the token's: larger or equal; after it: larger (the filling of a short group never is)
            my.above += count_above<DT, kVecs>(u, v0 > tokv ? xt : xt_below);
        } else if (gm >= xt) {
#pragma unroll
            for (int q = 0; q < kVecs; ++q) {
                const int v = v0 + q * kThreads;
                if (v >= nvec) break;
                if (v == tokv) {
#pragma unroll
                    for (int e = 0; e < EPV; ++e) {
                        const float x = element<DT>(u[q], e);
                        my.above += x > xt || (x == xt && first + v * EPV + e < tok);
                    }
                } else {
                    // nothing is below -inf: every entry before such a token is above it
                    my.above += v < tokv && xt == -INFINITY ? EPV : count_above<DT, 1>(u + q, v < tokv ? xt_below : xt);
                }
            }
        }
        if ((fmaxf(gm, kFloor) - my.m) * c > 4.0f) {
            const Part up{fmaxf(gm, kFloor), 0.0f, 0.0f, 0};
            join(my, up, c);
        }
        const uint64_t m2 = f2_pack(-my.m, -my.m);
        // Sums of the group. Without the clamp first: y is then -inf for entries of -inf (or
        // overflows), and y 2^y a NaN; only such a group is summed again with the clamp
        // (vectors of a masked vocabulary, the row's last group).
        float gs, ge;
        auto sums = [&](bool clamp) {
            uint64_t s2 = 0ull, e2 = 0ull;
#pragma unroll
            for (int q = 0; q < kVecs; ++q) {
                const uint32_t w[4] = {u[q].x, u[q].y, u[q].z, u[q].w};
#pragma unroll
                for (int i = 0; i < EPV / 2; ++i) {
                    float a, b;
                    if (DT == 1) {
                        a = __uint_as_float(w[i] << 16);
                        b = __uint_as_float(w[i] & 0xffff0000u);
                    } else {
                        a = __uint_as_float(w[2 * i]);
                        b = __uint_as_float(w[2 * i + 1]);
                    }
                    uint64_t y = f2_mul(f2_add(f2_pack(a, b), m2), c2);
                    if (clamp) y = f2_pack(max_nan(f2_lo(y), kFloor), max_nan(f2_hi(y), kFloor));
                    const uint64_t p = f2_pack(ex2_approx(f2_lo(y)), ex2_approx(f2_hi(y)));
                    s2 = f2_add(s2, p);
                    e2 = f2_fma(y, p, e2);
                }
            }
            gs = f2_lo(s2) + f2_hi(s2);
            ge = f2_lo(e2) + f2_hi(e2);
        };
        sums(false);
        if (ge != ge) sums(true);
        my.s += gs;
        my.e += ge;
    };
    for (int ch = 0; ch < nch; ++ch) {
        uint4 u[kVecs];
        load(ch, u);
        group(ch, u);
    }
    // ---- this CTA's sums ----
    float wmx = top;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) wmx = fmaxf(wmx, __shfl_xor_sync(0xffffffffu, wmx, o));
    join_lanes<5>(my, c);
    if (lane == 0) {
        sm.wpart[warp] = my;
        sm.wmax[warp] = wmx;
    }
    if (k > 0) {
        // tau: the k-th largest of the threads' maxima (0: fewer threads hold elements)
        uint32_t v = tid < nvec ? f2o(top) : 0u;
#pragma unroll
        for (int size = 2; size <= 32; size <<= 1)  // descending bitonic sort over the warp
#pragma unroll
            for (int s = size >> 1; s > 0; s >>= 1) {
                const uint32_t o = __shfl_xor_sync(0xffffffffu, v, s);
                v = (((lane & s) == 0) == ((lane & size) == 0)) ? max(o, v) : min(o, v);
            }
        if (lane < k) sm.wtop[lane * kWarps + warp] = v;  // the warps' largest, then their second, ..
        __syncthreads();
        if (tid < kWarps * k) {
            const uint32_t x = sm.wtop[tid];
            if (x != 0u) {
                int r = 0;  // values at or above x: tau is the largest x that k values reach
                const uint4* w4 = reinterpret_cast<const uint4*>(sm.wtop);
#pragma unroll 4
                for (int i = 0; i < kWarps * k / 4; ++i) {
                    const uint4 o = w4[i];
                    r += (o.x >= x) + (o.y >= x) + (o.z >= x) + (o.w >= x);
                }
                if (r >= k) atomicMax(&sm.tau, x);
            }
        }
        __syncthreads();
        const uint32_t tau = sm.tau;
        // every element >= tau of the groups that reach it
        auto hot = [&](int ch) -> bool {
            const uint32_t g = DT == 1 ? static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(gmax_raw)[ch * kThreads + tid]) << 16
                                       : reinterpret_cast<const uint32_t*>(gmax_raw)[ch * kThreads + tid];
            return g != 0u && g >= (DT == 1 ? tau & 0xffff0000u : tau);
        };
        // The groups are listed first and their vectors then dealt over the threads, so that
        // all are read at once. (Each thread reading its own groups, one vector after the
        // other, took a third of the kernel's time.)
        for (int ch = 0; ch < nch; ++ch) {
            if (!hot(ch)) continue;
            const int at = atomicAdd(&sm.ngroups, 1);
            if (at < kGroups) sm.groups[at] = static_cast<uint32_t>(ch * kThreads + tid);
        }
        __syncthreads();
        const int ng = sm.ngroups;
        if (ng <= kGroups) {
            for (int i = tid; i < ng * kVecs; i += kThreads) {
                const int at = static_cast<int>(sm.groups[i / kVecs]);
                const int v = (at / kThreads * kVecs + i % kVecs) * kThreads + at % kThreads;
                if (v >= nvec) continue;
                const uint4 u = ld_prior(vec + v);
#pragma unroll
                for (int e = 0; e < EPV; ++e) {
                    const float x = element<DT>(u, e);
                    if (x == x && f2o(x) >= tau) {
                        const int key = atomicAdd(&sm.nkeys, 1);
                        if (key < kKeys) sm.keys[key] = make_key(x, static_cast<uint32_t>(first + v * EPV + e));
                    }
                }
            }
        }
        __syncthreads();
        const int nk = ng <= kGroups ? sm.nkeys : kKeys + 1;
        if (nk <= kKeys) {
            for (int i = tid; i < nk; i += kThreads) {
                const unsigned long long key = sm.keys[i];
                int r = 0;
#pragma unroll 4
                for (int o = 0; o < nk; ++o) r += sm.keys[o] > key;
                if (r < k) sm.ctop[r] = key;
            }
        } else {  // many equal values at the top: k rounds, each the largest key below the last
            uint64_t prev = ~0ull;
            for (int r = 0; r < k; ++r) {
                uint64_t best = 0;
                for (int ch = 0; ch < nch; ++ch) {
                    if (!hot(ch)) continue;
                    for (int q = 0; q < kVecs; ++q) {
                        const int v = (ch * kVecs + q) * kThreads + tid;
                        if (v >= nvec) break;
                        const uint4 u = ld_prior(vec + v);
#pragma unroll
                        for (int e = 0; e < EPV; ++e) {
                            const float x = element<DT>(u, e);
                            const uint64_t key = x == x ? make_key(x, static_cast<uint32_t>(first + v * EPV + e)) : 0ull;
                            if (key < prev && key > best) best = key;
                        }
                    }
                }
                best = warp_max_u64(best);
                __syncthreads();
                if (lane == 0) sm.red[warp] = best;
                __syncthreads();
                for (int i = 0; i < kWarps; ++i) best = sm.red[i] > best ? sm.red[i] : best;
                if (tid == 0) sm.ctop[r] = best;
                prev = best;
                if (best == 0ull) break;  // uniform
            }
        }
    }
    __syncthreads();
    // ---- the row's results in the cluster's leader ----
    cg::cluster_group cluster = cg::this_cluster();
    if (cpr > 1) cluster_started_wait();
    Shared* lead = cpr > 1 ? cluster.map_shared_rank(&sm, 0) : &sm;
    if (tid < kMaxTopK) lead->rtop[rank * kMaxTopK + tid] = sm.ctop[tid];
    if (warp == 0) {
        static_assert(kWarps == 8, "three steps");
        Part p = sm.wpart[lane & 7];
        float m = sm.wmax[lane & 7];
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        join_lanes<3>(p, c);
        if (lane == 0) {
            lead->rpart[rank] = p;
            lead->rmax[rank] = m;
        }
    }
    if (cpr > 1) {
        cluster.sync();
        if (rank != 0) return;
    } else {
        __syncthreads();
    }
    Part p = sm.rpart[0];
    float m = sm.rmax[0];
    for (int i = 1; i < cpr; ++i) {
        join(p, sm.rpart[i], c);
        m = fmaxf(m, sm.rmax[i]);
    }
    if (m <= kFloor && m > -INFINITY) {
        // A row with nothing above the floor (a mask of the type's lowest value everywhere):
        // the clamp hides its differences, so the leader sums it again as it is.
        float s = 0.0f, e = 0.0f;
        for (int v = tid; v < a.V / EPV; v += kThreads) {
            const uint4 u = ld_prior(reinterpret_cast<const uint4*>(row) + v);
#pragma unroll
            for (int i = 0; i < EPV; ++i) {
                const float y = (element<DT>(u, i) - m) * c, w = ex2_approx(y);
                s += w;
                e += w > 0.0f ? y * w : 0.0f * w;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, o);
            e += __shfl_xor_sync(0xffffffffu, e, o);
        }
        __syncthreads();
        if (lane == 0) sm.wpart[warp] = Part{0.0f, s, e, 0};
        __syncthreads();
        p.m = m;
        p.s = p.e = 0.0f;
        for (int i = 0; i < kWarps; ++i) {
            p.s += sm.wpart[i].s;
            p.e += sm.wpart[i].e;
        }
    }
    const float ln2 = 0.693147180559945309417f, lns = logf(p.s);
    auto ln_p = [&](float x) -> float { return (x - p.m) / a.temperature - lns; };
    const bool bad = !(p.s > 0.0f) || !isfinite(p.s) || m == -INFINITY;
    if (tid == 0) {
        if (bad) raise_status(a.status, kDevNonFinite);
        a.logprob[entry] = bad ? NAN : ln_p(xt);
        if (a.entropy) a.entropy[entry] = bad ? NAN : lns - ln2 * (p.e / p.s);
        if (a.rank) a.rank[entry] = bad ? -1 : p.above;
    }
    if (bad) {  // NaN entries have no key: the alternatives of padding instead of what was there
        if (tid < k) {
            a.alt_ids[static_cast<size_t>(entry) * k + tid] = -1;
            a.alt_logprobs[static_cast<size_t>(entry) * k + tid] = NAN;
        }
        return;
    }
    if (tid < cpr * kMaxTopK && k > 0) {
        const uint64_t key = sm.rtop[tid];
        int r = tid;  // a single CTA's are in order
        if (cpr > 1 && key != 0ull) {
            r = 0;
            for (int i = 0; i < cpr * kMaxTopK; ++i) r += sm.rtop[i] > key;
        }
        if (key != 0ull && r < k) {
            a.alt_ids[static_cast<size_t>(entry) * k + r] = static_cast<int32_t>(key_id(key));
            a.alt_logprobs[static_cast<size_t>(entry) * k + r] = ln_p(key_val(key));
        }
    }
    if (tid < k && tid >= a.V) {  // alternatives past the row's entries
        a.alt_ids[static_cast<size_t>(entry) * k + tid] = -1;
        a.alt_logprobs[static_cast<size_t>(entry) * k + tid] = -INFINITY;
    }
}

template <int DT>
cudaError_t launch(const LogprobArgs& a, cudaStream_t stream) {
    constexpr int ES = DT == 1 ? 2 : 4;
    // CTAs per row: enough to fill the machine (four CTAs per SM) with the
    // entries there are, at least one chunk each
    const int max_cpr = std::max(1, std::min<int>(kMaxChunks, static_cast<int>(static_cast<long>(a.V) * ES / kChunkBytes)));
    int cpr = 1;
    while (cpr * 2 <= max_cpr && static_cast<long>(a.n) * cpr < 152 * 4) cpr *= 2;
    const int seg = row_seg_elems(a.V, ES, cpr);
    const int nch = (seg * ES + kChunkBytes - 1) / kChunkBytes;
    const int smem = a.n_alt > 0 ? nch * kThreads * (DT == 1 ? 2 : 4) : 0;
    auto kernel = token_logprobs_kernel<DT>;
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.n) * cpr);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cpr;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    count_launch();
    return cudaLaunchKernelEx(&cfg, kernel, a, cpr, seg, kLog2e / a.temperature);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, int dtype, cudaStream_t stream) {
    return dtype == 1 ? launch<1>(a, stream) : launch<0>(a, stream);
}

}  // namespace eagle
