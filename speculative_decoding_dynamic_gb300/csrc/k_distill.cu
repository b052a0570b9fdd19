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
// arithmetic); the listed entries are taken out of it, each CTA sums
// exp((z - m) / T) over the rest of its segment, and one exchange of (m, sum)
// through distributed shared memory gives every CTA the row's sums. The rest is
// summed by itself, so that a draft that is sure of the listed ids loses
// nothing of q_R to cancellation.

#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "eagle_internal.cuh"
#include "eagle_ws.h"
#include "quant_ptx.cuh"
#include "quant_ws.h"

namespace eagle {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSegBytes = 65536;  // of a row in a CTA's shared memory
constexpr int kCopyBytes = 16384;
constexpr float kLog2e = 1.4426950408889634f;
static_assert(kDistillMaxTop <= kThreads, "a thread for each listed id");

struct Part {  // a CTA's share of the row outside the list
    float m, s;
    int bad;  // a DeviceError, 0 = none
};
struct Shared {
    alignas(8) uint64_t bar;
    float redf[kWarps];
    double redd[kWarps];
    float wm[kWarps], ws[kWarps];
    int bad;
    Part part[kMaxChunks];  // of all CTAs of the cluster
};

template <int DT>
__device__ __forceinline__ float load1(const void* row, int i) {
    if (DT == 1)
        return __uint_as_float(static_cast<uint32_t>(ld_prior(static_cast<const unsigned short*>(row) + i)) << 16);
    return ld_prior(static_cast<const float*>(row) + i);
}
template <int DT>
__device__ __forceinline__ void unpack(const uint4& u, float (&x)[DT == 1 ? 8 : 4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (DT == 1) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            x[i] = __uint_as_float(w[i]);
        }
    }
}

__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) v = fmaxf(v, red[i]);
    return v;
}
template <typename T>
__device__ __forceinline__ T block_sum(T v, T* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) v += red[i];
    return v;
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 3) distill_kernel(DistillArgs a, int cpr, int seg, float c) {
    extern __shared__ __align__(128) unsigned char row_smem[];
    __shared__ Shared sm;
    constexpr int ES = DT == 1 ? 2 : 4;
    constexpr int EPV = 16 / ES;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
    const float w = a.row_weight ? ld_prior(a.row_weight + row) : 1.0f;
    // ---- the target's list: thread t holds entry t ----
    int id = -1;
    float t = -INFINITY;
    if (tid < a.n_top) {
        id = ld_prior(a.ids + static_cast<size_t>(row) * a.n_top + tid);
        t = ld_prior(a.teacher + static_cast<size_t>(row) * a.n_top + tid);
    }
    const bool whole = a.teacher_lse == nullptr;  // the list is the whole distribution
    const bool listed = __syncthreads_or(id >= 0);
    if (w == 0.0f || (whole && !listed)) {  // no weight, or nothing to learn: uniform over the cluster
        if (grad)
            for (int v = tid; v < nvec; v += kThreads) grad[v] = make_uint4(0u, 0u, 0u, 0u);
        if (rank == 0 && tid == 0) a.loss[row] = 0.0f;
        return;
    }
    if (cpr > 1) cluster_started_arrive();
    if (tid == 0) {
        mbar_init(&sm.bar, 1);
        fence_mbar_init();
        sm.bad = isfinite(w) ? 0 : kDevNonFinite;
    }
    __syncthreads();
    if (tid == 0) {
        mbar_arrive_expect_tx(&sm.bar, static_cast<uint32_t>(n) * ES);
        for (int off = 0; off < n * ES; off += kCopyBytes)
            bulk_g2s(row_smem + off, in + static_cast<size_t>(first) * ES + off,
                     static_cast<uint32_t>(min(kCopyBytes, n * ES - off)), &sm.bar);
    }
    int bad = 0;
    if (id >= a.V) {
        bad = kDevBadIndex;
        id = -1;
    }
    const bool on = id >= 0;
    const float z = on ? load1<DT>(in, id) : -INFINITY;  // the draft's logit there
    // the target's log-probabilities
    float lnp = -INFINITY, p = 0.0f;
    if (whole) {
        const float top = block_max(on ? t : -INFINITY, sm.redf);
        const float y = on ? (t - top) / a.temperature : -INFINITY;
        const float e = on ? expf(y) : 0.0f;
        const float total = block_sum(e, sm.redf);
        lnp = y - logf(total);
        if (!(total > 0.0f) || !isfinite(total)) bad = kDevNonFinite;
    } else {
        const float lse = ld_prior(a.teacher_lse + row);
        lnp = t / a.temperature - lse;
        if (!isfinite(lse)) bad = kDevNonFinite;
    }
    if (on) p = expf(lnp);
    if (on && !(p < INFINITY)) bad = kDevNonFinite;
    const double psum = block_sum(static_cast<double>(p), sm.redd);
    const float r = whole ? 0.0f : static_cast<float>(fmax(0.0, 1.0 - psum));
    const float mass = whole ? 1.0f : static_cast<float>(psum) + r;
    // ---- the segment ----
    const bool arrived = mbar_wait_sleep(&sm.bar, 0);
    if (!arrived) bad = kDevTimeout;
    // An id listed twice: the last of its entries to write its number there finds another one.
    const bool mine = on && id >= first && id < first + n;
    if (arrived && mine) {
        if (DT == 1) reinterpret_cast<volatile uint16_t*>(row_smem)[id - first] = static_cast<uint16_t>(tid);
        else reinterpret_cast<volatile uint32_t*>(row_smem)[id - first] = static_cast<uint32_t>(tid);
    }
    __syncthreads();
    if (arrived && mine) {
        const uint32_t who = DT == 1 ? reinterpret_cast<volatile uint16_t*>(row_smem)[id - first]
                                     : reinterpret_cast<volatile uint32_t*>(row_smem)[id - first];
        if (who != static_cast<uint32_t>(tid)) bad = kDevBadIndex;
    }
    __syncthreads();
    if (arrived && mine) {  // the list's entries leave the segment
        if (DT == 1) reinterpret_cast<uint16_t*>(row_smem)[id - first] = 0xff80u;
        else reinterpret_cast<uint32_t*>(row_smem)[id - first] = 0xff800000u;
    }
    if (bad) atomicMax(&sm.bad, bad);
    __syncthreads();
    const uint4* vec = reinterpret_cast<const uint4*>(row_smem);
    float m = -INFINITY;
    for (int v = tid; v < nvec; v += kThreads) {
        float x[EPV];
        unpack<DT>(vec[v], x);
#pragma unroll
        for (int i = 0; i < EPV; ++i) m = fmaxf(m, x[i]);
    }
    float s = 0.0f;
    const float m0 = m == -INFINITY ? 0.0f : m;  // nothing but -inf: every term is 0
    for (int v = tid; v < nvec; v += kThreads) {
        float x[EPV];
        unpack<DT>(vec[v], x);
        float part = 0.0f;
#pragma unroll
        for (int i = 0; i < EPV; ++i) part += ex2_approx((x[i] - m0) * c);
        s += part;
    }
    // joined over the CTA
    auto join = [&](float& am, float& as, float bm, float bs) {
        const float M = fmaxf(am, bm), M0 = M == -INFINITY ? 0.0f : M;
        as = as * ex2_approx((am - M0) * c) + bs * ex2_approx((bm - M0) * c);
        am = M;
    };
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, m, o), os = __shfl_xor_sync(0xffffffffu, s, o);
        join(m, s, om, os);
    }
    if (lane == 0) {
        sm.wm[warp] = m;
        sm.ws[warp] = s;
    }
    __syncthreads();
    m = sm.wm[0];
    s = sm.ws[0];
    for (int i = 1; i < kWarps; ++i) join(m, s, sm.wm[i], sm.ws[i]);
    // ---- joined over the cluster ----
    cg::cluster_group cluster = cg::this_cluster();
    if (cpr > 1) cluster_started_wait();
    if (tid < cpr) {
        Part* to = cpr > 1 ? cluster.map_shared_rank(&sm.part[rank], tid) : &sm.part[rank];
        *to = Part{m, s, sm.bad};
    }
    if (cpr > 1) cluster.sync();
    else __syncthreads();
    int fault = sm.part[0].bad;
    m = sm.part[0].m;
    float sr = sm.part[0].s;
    for (int i = 1; i < cpr; ++i) {
        join(m, sr, sm.part[i].m, sm.part[i].s);
        fault = max(fault, sm.part[i].bad);
    }
    const float ztop = block_max(z, sm.redf);
    const float M = fmaxf(m, ztop), M0 = M == -INFINITY ? 0.0f : M;
    sr *= ex2_approx((m - M0) * c);
    const float e = on ? ex2_approx((z - M0) * c) : 0.0f;
    const float total = sr + block_sum(e, sm.redf);
    const float lns = logf(total);
    // a NaN among the list's logits is in e, one of the rest in sr; a maximum of +inf makes them NaN
    if (fault == 0 && (!(total > 0.0f) || !isfinite(total))) fault = kDevNonFinite;
    const bool rest = r > 0.0f && sr > 0.0f;
    if (rank == 0) {
        // p ln p is 0 where p is; a listed id that the draft rules out makes the loss infinite
        float term = on && p > 0.0f ? p * (lnp - ((z - M0) / a.temperature - lns)) : 0.0f;
        term = block_sum(term, sm.redf);
        if (tid == 0) {
            if (rest) term += r * (logf(r) - (logf(sr) - lns));
            if (fault) raise_status(a.status, fault);
            a.loss[row] = fault ? NAN : w * term;
        }
    }
    if (grad == nullptr) return;
    if (fault) {
        for (int v = tid; v < nvec; v += kThreads) grad[v] = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    const float wt = w / a.temperature;
    const float factor = wt * (mass / total - (rest ? r / sr : 0.0f));
    for (int v = tid; v < nvec; v += kThreads) {
        float x[EPV];
        unpack<DT>(vec[v], x);
#pragma unroll
        for (int i = 0; i < EPV; ++i) x[i] = ex2_approx((x[i] - M0) * c) * factor;
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (DT == 1) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[(2 * i) % EPV], x[(2 * i + 1) % EPV]);
                o[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                o[i] = __float_as_uint(x[i]);
            }
        }
        grad[v] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    __syncthreads();  // the list's entries after the vectors that hold them
    if (mine) {
        const float g = wt * (mass * (e / total) - p);
        if (DT == 1) reinterpret_cast<__nv_bfloat16*>(grad)[id - first] = __float2bfloat16_rn(g);
        else reinterpret_cast<float*>(grad)[id - first] = g;
    }
}

template <int DT>
cudaError_t launch(const DistillArgs& a, cudaStream_t stream) {
    constexpr int ES = DT == 1 ? 2 : 4;
    // CTAs of a row: as many as hold it, more where there are few rows
    int cpr = 1;
    while (cpr < kMaxChunks && row_seg_elems(a.V, ES, cpr) * ES > kMaxSegBytes) cpr *= 2;
    while (cpr < kMaxChunks && static_cast<long>(a.rows) * cpr < 152 * 3 && row_seg_elems(a.V, ES, cpr * 2) * ES >= kCopyBytes) cpr *= 2;
    const int seg = row_seg_elems(a.V, ES, cpr);
    const int smem = seg * ES;
    auto kernel = distill_kernel<DT>;
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * cpr);
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

cudaError_t launch_distill(const DistillArgs& a, int dtype, cudaStream_t stream) {
    return dtype == 1 ? launch<1>(a, stream) : launch<0>(a, stream);
}

}  // namespace eagle
