// Device helpers shared by the kernels on quantised operands. Not part of the public ABI.
#pragma once

#include "eagle_internal.cuh"

namespace eagle {

// An ordinary load of data that an earlier kernel of the stream may have
// written. Not __ldg: that promises that nothing writes the data while this
// grid runs, and a grid launched with programmatic serialisation runs before
// the earlier kernel has ended (pdl_wait_prior), so its loads could be taken
// from before the wait.
template <typename V>
__device__ __forceinline__ V ld_prior(const V* p) {
    return *p;
}

// The power of two that brings a row's largest element amax into [2^to, 2^(to + 1)).
__device__ __forceinline__ float pow2_to(float amax, int to) {
    const int e = static_cast<int>(__float_as_uint(amax) >> 23);  // biased; 0 for zero and subnormals
    const int f = to + 254 - e;                                   // biased exponent of the scale
    return __uint_as_float(static_cast<uint32_t>(max(1, min(f, 253))) << 23);
}

// One look at an mbarrier phase, without waiting.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// 16 bytes from / to shared memory by its 32-bit address (a pointer into
// dynamic shared memory that was aligned by hand is a generic one to the
// compiler, and generic loads are tracked like global ones).
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

}  // namespace eagle
