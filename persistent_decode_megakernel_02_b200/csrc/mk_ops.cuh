// mk_ops.cuh -- device helpers shared by the serving operators' kernels:
// 16-bit element types, packed conversions, the sequence lookup of packed
// rows, and the status word.  Device code only; not part of the public ABI.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mk_ops.h"
#include "mk_ptx.cuh"

namespace mk {

// Two 16-bit elements of a 32-bit word, widened; and back, each rounded to
// nearest even.
struct Bf16 {
    static constexpr bool kBf16 = true;
    static __device__ __forceinline__ float2 unpack(uint32_t w) { return make_float2(bf_lo(w), bf_hi(w)); }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};
struct Fp16 {
    static constexpr bool kBf16 = false;
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};

__device__ __forceinline__ void bad_value(int32_t *status) {
    if (status) *status = MK_ERR_INVALID;
}

// The sequence of packed row t: the largest s with cu[s] <= t (0 if none),
// found by a whole warp, 32 candidates a step.  Any cu gives an s in
// [0, n): callers check the row against that sequence's own bounds.
__device__ __forceinline__ int warp_find_seq(const int32_t *cu, int n, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n;   // the answer lies in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5;
        const int s = lo + lane * step;
        const unsigned le = __ballot_sync(0xffffffffu, s < hi && (lane == 0 || cu[s] <= t));
        // candidates are in order, so the ones at or below t come first
        const int last = 31 - __clz(le);
        lo += last * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

}  // namespace mk
