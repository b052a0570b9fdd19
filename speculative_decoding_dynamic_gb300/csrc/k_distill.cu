// The loss that trains a draft on its target's top logits, with its gradient
// (sm_103a): eagle_distill_loss.
//
// With z the draft's row, q = softmax(z / T), p the target's probabilities of
// its listed ids and r what they leave (0 where the list is taken for the whole
// distribution), q_R the draft's probability of everything else:
//   L       = sum p (ln p - ln q) + r (ln r - ln q_R)
//   dL/dz_j = (1/T) ((sum p + r) q_j - p_j)           j in the list
//           = (1/T) q_j ((sum p + r) - r / q_R)       elsewhere
// so outside the list the gradient is exp((z_j - M) / T) times one factor of the
// row, and only the list's own entries need p.
//
// Bound by HBM: a row is read once and its gradient written once. A row lies in
// the shared memory of a cluster of 1..8 CTAs (bulk copies, at most 64 KB a
// CTA, so that three CTAs share an SM and one's copies run behind another's
// arithmetic). The first warp takes the listed entries out of the row and then
// works out the target's side while the others sum exp((z - m) / T) over the
// rest, and one exchange of (m, sum) through distributed shared memory gives
// every CTA the row's sums. The rest is summed by itself and relative to its own
// largest logit m_R, so that a draft that is sure of the listed ids loses nothing
// of q_R to cancellation, and however far the rest lies below them nothing of it
// underflows: with s = sum over the rest of exp((z - m_R) / T), which is at least 1,
//   ln q_R  = (m_R - M) / T + ln s - ln total
//   dL/dz_j = (1/T) exp((z_j - m_R) / T) ((sum p + r) exp((m_R - M) / T) / total - r / s)
//
// Measured: 4096 fp32 rows of 32000 (983 MB) 161 us, 90% of HBM; 640 bf16 rows of
// 128256 (308 MB) 60 us, 76%: six waves of CTAs that run much in step; 10 rows 6.7
// us (5.5 where they lie in L2). The loss alone: 107, 42 and 5.7 us.

#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "eagle_internal.cuh"
#include "eagle_ws.h"
#include "quant_ptx.cuh"
#include "quant_ws.h"

namespace eagle {
namespace {

constexpr int kMaxWarps = 8;
constexpr int kMaxSegBytes = 65536;  // of a row in a CTA's shared memory
constexpr int kCopyBytes = 16384;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRuledOut = 0x1p20f;  // times T if that is above 1: a rest further under the row's top is masked, by -inf or a type's lowest value

struct Shared {
    alignas(8) uint64_t bar;
    float2 part[kMaxChunks * (kMaxWarps - 1)];  // (m, sum) of the rest, of each warp but the first of each CTA of the cluster
    int bad[kMaxChunks];                  // a DeviceError of each CTA, 0 = none
    float2 list;                          // (m, sum) of the listed entries
    float r, mass, psum;                  // what the list leaves; sum p + r; sum p
    int nothing;                          // a list of padding alone that is the whole distribution: no fault by itself
    int id[kDistillMaxTop];               // -1: padding, or no entry of the row
    float z[kDistillMaxTop], lnp[kDistillMaxTop];
};

template <int DT>
__device__ __forceinline__ float load1(const void* row, int i) {
    if (DT == 1)
        return __uint_as_float(static_cast<uint32_t>(ld_prior(static_cast<const unsigned short*>(row) + i)) << 16);
    return ld_prior(static_cast<const float*>(row) + i);
}
__device__ __forceinline__ __nv_bfloat162 bf2(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }
// The entries of 16 bytes as packed pairs.
template <int DT>
__device__ __forceinline__ void unpack(const uint4& u, uint64_t (&x)[DT == 1 ? 4 : 2]) {
    if (DT == 1) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i % (DT == 1 ? 4 : 2)] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    } else {
        x[0] = f2_pack(__uint_as_float(u.x), __uint_as_float(u.y));
        x[1] = f2_pack(__uint_as_float(u.z), __uint_as_float(u.w));
    }
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// ln x of a positive x: the exponent's part apart, so that the logarithm's rounding is that of a value below 0.41.
__device__ __forceinline__ double ln_fine(float x) {
    const bool small = x < 0x1p-60f;
    if (small) x *= 0x1p66f;  // (subnormals)
    const uint32_t b = __float_as_uint(x) - 0x3f3504f3u;  // (bits of sqrt(1/2): the rest is in [0.71, 1.41))
    const int e = (static_cast<int>(b) >> 23) - (small ? 66 : 0);
    return fma(static_cast<double>(e), 0.693147180559945309417, static_cast<double>(logf(__uint_as_float((b & 0x7fffffu) + 0x3f3504f3u))));
}

template <int DT>
__global__ void __launch_bounds__(kMaxWarps * 32, 3) distill_kernel(DistillArgs a, int cpr, int seg, int ahead, float c, double inv_t) {
    extern __shared__ __align__(128) unsigned char row_smem[];
    __shared__ Shared sm;
    constexpr int ES = DT == 1 ? 2 : 4;
    constexpr int EPV = 16 / ES;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads >> 5;
    const int row = blockIdx.x / cpr, rank = blockIdx.x % cpr;  // a cluster is cpr neighbouring CTAs
    pdl_launch_dependents();
    pdl_wait_prior();
    const int first = rank * seg;  // this CTA's elements [first, first + n)
    const int n = max(0, min(seg, a.V - first));
    const int nvec = n / EPV;
    const size_t row_bytes = static_cast<size_t>(a.V) * ES;
    const char* in = static_cast<const char*>(a.logits) + static_cast<size_t>(row) * row_bytes;
    uint4* grad = a.grad ? reinterpret_cast<uint4*>(static_cast<char*>(a.grad) + static_cast<size_t>(row) * row_bytes +
                                                    static_cast<size_t>(first) * ES)
                         : nullptr;
    // The first warp's lanes hold the target's list, 32 apart (all loads of a kind go out together)
    constexpr int kSlots = kDistillMaxTop / 32;
    int id[kSlots];
    float t[kSlots], lse = 0.0f;
    if (warp == 0) {
        const size_t at = static_cast<size_t>(row) * a.n_top;
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
            const int i = k * 32 + lane;
            id[k] = i < a.n_top ? ld_prior(a.ids + at + i) : -1;
            t[k] = i < a.n_top ? ld_prior(a.teacher + at + i) : -INFINITY;
        }
        if (a.teacher_lse) lse = ld_prior(a.teacher_lse + row);
    }
    const float w = a.row_weight ? ld_prior(a.row_weight + row) : 1.0f;
    if (w == 0.0f) {  // uniform over the cluster
        if (grad)
            for (int v = tid; v < nvec; v += threads) grad[v] = make_uint4(0u, 0u, 0u, 0u);
        if (rank == 0 && tid == 0) a.loss[row] = 0.0f;
        return;
    }
    if (cpr > 1) cluster_started_arrive();
    if (tid == 0) {
        mbar_init(&sm.bar, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(&sm.bar, static_cast<uint32_t>(n) * ES);
        for (int off = 0; off < n * ES; off += kCopyBytes)
            bulk_g2s(row_smem + off, in + static_cast<size_t>(first) * ES + off,
                     static_cast<uint32_t>(min(kCopyBytes, n * ES - off)), &sm.bar);
    }
    int bad = 0;
    float z[kSlots];
    if (warp == 0) {
        // ---- the list's entries leave the row ----
        __syncwarp();
        bad = isfinite(grad ? w / a.temperature : w) ? 0 : kDevNonFinite;  // (the gradient's factor)
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
            z[k] = -INFINITY;
            if (k * 32 >= a.n_top) continue;
            if (id[k] >= a.V) {
                bad = kDevBadIndex;
                id[k] = -1;
            }
            if (id[k] >= 0) z[k] = load1<DT>(in, id[k]);  // the draft's logit there
        }
        if (mbar_wait_sleep(&sm.bar, 0)) {
            // An id listed twice: the last of its entries to write its number there finds another one
            auto slot = [&](int k) -> int {  // where entry k lies in this CTA's segment, -1: not there
                const int at = id[k] - first;
                return k * 32 < a.n_top && id[k] >= 0 && at >= 0 && at < n ? at : -1;
            };
            volatile uint16_t* row16 = reinterpret_cast<volatile uint16_t*>(row_smem);
            volatile uint32_t* row32 = reinterpret_cast<volatile uint32_t*>(row_smem);
#pragma unroll
            for (int k = 0; k < kSlots; ++k) {
                const int at = slot(k);
                if (at < 0) continue;
                if (DT == 1) row16[at] = static_cast<uint16_t>(k * 32 + lane);
                else row32[at] = static_cast<uint32_t>(k * 32 + lane);
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < kSlots; ++k) {
                const int at = slot(k);
                if (at < 0) continue;
                if ((DT == 1 ? static_cast<uint32_t>(row16[at]) : row32[at]) != static_cast<uint32_t>(k * 32 + lane)) bad = kDevBadIndex;
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < kSlots; ++k) {
                const int at = slot(k);
                if (at < 0) continue;
                if (DT == 1) row16[at] = 0xff80u;
                else row32[at] = 0xff800000u;
            }
        } else {
            bad = kDevTimeout;
        }
    }
    // A CTA that starts when this one ends finds its row on its way or in L2: HBM reads go on while the CTAs of an SM,
    // which run much in step, add up and store.
    if (tid == 32 && row + ahead < a.rows && (a.row_weight == nullptr || ld_prior(a.row_weight + row + ahead) != 0.0f))
        for (int off = 0; off < n * ES; off += kCopyBytes)
            prefetch_l2(in + static_cast<size_t>(ahead) * row_bytes + static_cast<size_t>(first) * ES + off,
                        static_cast<uint32_t>(min(kCopyBytes, n * ES - off)));
    __syncthreads();
    mbar_try_wait(&sm.bar, 0);  // done: every thread that reads what was copied has seen it
    const uint4* vec = reinterpret_cast<const uint4*>(row_smem);
    const uint64_t c2 = f2_pack(c, c);
    float m = -INFINITY, s = 0.0f;
    if (warp == 0) {
        // ---- the target's side ----
        const bool whole = a.teacher_lse == nullptr;  // the list is the whole distribution
        bool any = false;
        float top = -INFINITY, ztop = -INFINITY;
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
            any = any || id[k] >= 0;
            if (id[k] >= 0) top = fmaxf(top, t[k]);
            ztop = fmaxf(ztop, z[k]);
        }
        any = __any_sync(0xffffffffu, any);
        // a list whose logits are all -inf (or NaN) is no distribution, with an lse neither
        if (any && !__any_sync(0xffffffffu, top > -INFINITY)) bad = max(bad, static_cast<int>(kDevNonFinite));
        ztop = warp_max(ztop);
        const float z0 = ztop == -INFINITY ? 0.0f : ztop;
        float shift = lse;
        if (whole) {
            top = warp_max(top);
            float total = 0.0f;
#pragma unroll
            for (int k = 0; k < kSlots; ++k) {
                if (k * 32 >= a.n_top) continue;
                t[k] = t[k] - top;
                if (id[k] >= 0) total += expf(t[k] / a.temperature);
            }
            total = warp_sum(total);
            shift = logf(total);
        }
        if ((any || !whole) && !isfinite(shift)) bad = max(bad, static_cast<int>(kDevNonFinite));
        float zsum = 0.0f, psum = 0.0f, low = 0.0f;  // (sum p and what its roundings lost: 1 - sum p is of that size)
        auto add = [&](float p) {
            const float u = psum + p, q = u - psum;
            low += (psum - (u - q)) + (p - q);
            psum = u;
        };
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
            const int i = k * 32 + lane;
            if (k * 32 >= a.n_top) continue;
            const bool on = id[k] >= 0;
            // (t / T and the lse nearly cancel: their difference is rounded once)
            const float lnp = on ? static_cast<float>(fma(static_cast<double>(t[k]), inv_t, -static_cast<double>(shift))) : -INFINITY;
            const float p = on ? expf(lnp) : 0.0f;
            if (!(p < INFINITY)) bad = max(bad, static_cast<int>(kDevNonFinite));
            add(p);
            if (on) zsum += ex2_approx((z[k] - z0) * c);  // a NaN or +inf logit makes it NaN
            if (i < a.n_top) {
                sm.id[i] = id[k];
                sm.z[i] = z[k];
                sm.lnp[i] = lnp;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            low += __shfl_xor_sync(0xffffffffu, low, o);
            add(__shfl_xor_sync(0xffffffffu, psum, o));
            zsum += __shfl_xor_sync(0xffffffffu, zsum, o);
        }
        bad = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(bad)));
        if (lane == 0) {
            // (lanes differ in `low` by what their own last sums lost: far below what matters)
            const float r = whole ? 0.0f : fmaxf(0.0f, (1.0f - psum) - low);
            sm.r = r;
            sm.psum = psum;
            sm.mass = whole ? 1.0f : psum + r;
            sm.list = make_float2(ztop, zsum);
            sm.nothing = whole && !any;
            sm.bad[rank] = bad;
        }
        __syncwarp();
    } else {
        // ---- the rest: this warp's largest entry, then its sum relative to it (no reference to agree on first) ----
        const int t0 = tid - 32, step = threads - 32;
        if (DT == 1) {
            __nv_bfloat162 top = __floats2bfloat162_rn(-INFINITY, -INFINITY);
            for (int v = t0; v < nvec; v += step) {
                const uint4 u = vec[v];
                top = __hmax2(top, __hmax2(__hmax2(bf2(u.x), bf2(u.y)), __hmax2(bf2(u.z), bf2(u.w))));
            }
            m = fmaxf(__low2float(top), __high2float(top));
        } else {
            for (int v = t0; v < nvec; v += step) {
                const uint4 u = vec[v];
                m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w))));
            }
        }
        m = warp_max(m);
        const float m0 = m == -INFINITY ? 0.0f : m;  // nothing but -inf: every term is 0
        const uint64_t minus = f2_pack(-m0, -m0);
        uint64_t s2[2] = {0ull, 0ull};
        for (int v = t0; v < nvec; v += step) {
            uint64_t x[EPV / 2];
            unpack<DT>(vec[v], x);
#pragma unroll
            for (int i = 0; i < EPV / 2; ++i) {
                const uint64_t y = f2_mul(f2_add(x[i], minus), c2);
                s2[i & 1] = f2_add(s2[i & 1], f2_pack(ex2_approx(f2_lo(y)), ex2_approx(f2_hi(y))));
            }
        }
        const uint64_t u = f2_add(s2[0], s2[1]);
        s = warp_sum(f2_lo(u) + f2_hi(u));
    }
    // ---- over the cluster ----
    const int nparts = warps - 1;  // of a CTA
    cg::cluster_group cluster = cg::this_cluster();
    if (cpr > 1) {
        cluster_started_wait();
        if (warp > 0 && lane < cpr) *cluster.map_shared_rank(&sm.part[rank * nparts + warp - 1], lane) = make_float2(m, s);
        if (warp == 0 && lane < cpr) *cluster.map_shared_rank(&sm.bad[rank], lane) = bad;
        cluster.sync();
    } else {
        if (warp > 0 && lane == 0) sm.part[warp - 1] = make_float2(m, s);
        __syncthreads();
    }
    // the parts over their largest m, two a lane at most
    static_assert(kMaxChunks * (kMaxWarps - 1) <= 64, "two parts a lane");
    const float2 none = make_float2(-INFINITY, 0.0f);
    const float2 p0 = lane < cpr * nparts ? sm.part[lane] : none, p1 = lane + 32 < cpr * nparts ? sm.part[lane + 32] : none;
    const float mr = warp_max(fmaxf(p0.x, p1.x)), mr0 = mr == -INFINITY ? 0.0f : mr;  // the rest's largest (none: 0)
    const float M = fmaxf(mr, sm.list.x), M0 = M == -INFINITY ? 0.0f : M;
    const float sr = warp_sum(p0.y * ex2_approx((p0.x - mr0) * c) + p1.y * ex2_approx((p1.x - mr0) * c));  // relative to it
    const float down = ex2_approx((mr - M0) * c), rest = sr * down;  // relative to M: 0 where there is none or far below
    const float listed = sm.list.y * ex2_approx((sm.list.x - M0) * c), total = rest + listed, r = sm.r;
    int fault = lane < cpr ? sm.bad[lane] : 0;
    fault = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(fault)));
    // a NaN is in one of the sums, a maximum of +inf makes them NaN
    if (!(total > 0.0f) || !isfinite(total)) fault = max(fault, static_cast<int>(kDevNonFinite));
    const bool nothing = sm.nothing != 0, leaves = r > 0.0f && mr > -INFINITY && M0 - mr <= kRuledOut * fmaxf(1.0f, a.temperature);
    const float wt = w / a.temperature;
    if (rank == 0 && warp == 0) {
        // The loss is a difference of logarithms, often far smaller than they are: differences in 64 bits, of logarithms
        // that are within 2^-25 (beside the other warps' gradient)
        const double lns = ln_fine(total);
        float term = 0.0f;
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
            const int i = k * 32 + lane;
            if (i >= a.n_top) continue;
            // p ln p is 0 where p is; a listed id that the draft rules out makes the loss infinite
            const float lnp = sm.lnp[i], p = expf(lnp);
            const double lnq = (static_cast<double>(z[k]) - static_cast<double>(M0)) * inv_t - lns;
            if (id[k] >= 0 && p > 0.0f) term += p * static_cast<float>(static_cast<double>(lnp) - lnq);
        }
        term = warp_sum(term);
        if (lane == 0) {
            if (leaves) {
                // ln r and ln q_R from the list's side where that is the smaller part
                const float ps = sm.psum;
                const double lnr = ps < 0.5f ? static_cast<double>(log1pf(-ps)) : ln_fine(r);
                const double lnqr = listed < rest ? static_cast<double>(log1pf(-listed / total))
                                                  : (static_cast<double>(mr) - static_cast<double>(M0)) * inv_t + ln_fine(sr) - lns;
                term += r * static_cast<float>(lnr - lnqr);
            }
            if (fault) raise_status(a.status, fault);
            a.loss[row] = fault ? NAN : nothing ? 0.0f : w * term;
        }
    }
    if (grad == nullptr) return;
    if (fault || nothing) {
        for (int v = tid; v < nvec; v += threads) grad[v] = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    // Of exp((z - mr) / T): (sum p + r) down / total - r / sr, with sum p + r - r total / rest = sum p - r listed / rest
    // where the list is the smaller part
    const float share = down / total;
    const float factor = wt * (!leaves ? sm.mass * share : listed < rest ? (sm.psum - r * (listed / rest)) * share : sm.mass * share - r / sr);
    const uint64_t minus = f2_pack(-mr0, -mr0), f2 = f2_pack(factor, factor);
    if (warp > 0) {
        for (int v = tid - 32; v < nvec; v += threads - 32) {
            uint64_t x[EPV / 2];
            unpack<DT>(vec[v], x);
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < EPV / 2; ++i) {
                const uint64_t y = f2_mul(f2_add(x[i], minus), c2);
                const uint64_t g = f2_mul(f2_pack(ex2_approx(f2_lo(y)), ex2_approx(f2_hi(y))), f2);
                if (DT == 1) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(f2_lo(g), f2_hi(g));
                    o[i] = *reinterpret_cast<const uint32_t*>(&h);
                } else {
                    o[2 * (i & 1)] = __float_as_uint(f2_lo(g));
                    o[2 * (i & 1) + 1] = __float_as_uint(f2_hi(g));
                }
            }
            grad[v] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    __syncthreads();  // the list's entries after the vectors that hold them
    if (warp == 0) {
        for (int i = lane; i < a.n_top; i += 32) {
            const int at = sm.id[i] - first;
            if (sm.id[i] < 0 || at < 0 || at >= n) continue;
            const float g = wt * (sm.mass * (ex2_approx((sm.z[i] - M0) * c) / total) - expf(sm.lnp[i]));
            if (DT == 1) reinterpret_cast<__nv_bfloat16*>(grad)[at] = __float2bfloat16_rn(g);
            else reinterpret_cast<float*>(grad)[at] = g;
        }
    }
}

template <int DT>
cudaError_t launch(const DistillArgs& a, cudaStream_t stream) {
    constexpr int ES = DT == 1 ? 2 : 4;
    // CTAs of a row: as many as hold it, more where there are fewer than SMs (100 rows of 128256 bf16 entries: four a row
    // 14.6 us, eight 17.2)
    int cpr = 1;
    while (cpr < kMaxChunks && row_seg_elems(a.V, ES, cpr) * ES > kMaxSegBytes) cpr *= 2;
    while (cpr < kMaxChunks && static_cast<long>(a.rows) * cpr < 152 && row_seg_elems(a.V, ES, cpr * 2) * ES >= kCopyBytes) cpr *= 2;
    const int seg = row_seg_elems(a.V, ES, cpr);
    const int smem = seg * ES;
    const int warps = smem > 16384 ? kMaxWarps : smem > 4096 ? 4 : 2;  // of short rows more share an SM
    // rows at once, as far as shared memory, threads and registers decide it
    const int at_once = std::min({(226 * 1024) / (smem + static_cast<int>(sizeof(Shared)) + 1024), 2048 / (warps * 32), 24, 24 / warps});
    const int ahead = std::max(1, 38 * std::max(1, at_once) / cpr);  // a quarter of them: half and all were slower
    auto kernel = distill_kernel<DT>;
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * cpr);
    cfg.blockDim = dim3(static_cast<unsigned>(warps * 32));
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
    return cudaLaunchKernelEx(&cfg, kernel, a, cpr, seg, ahead, kLog2e / a.temperature, 1.0 / static_cast<double>(a.temperature));
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, int dtype, cudaStream_t stream) {
    return dtype == 1 ? launch<1>(a, stream) : launch<0>(a, stream);
}

}  // namespace eagle
