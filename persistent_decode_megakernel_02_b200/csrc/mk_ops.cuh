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

// 2^x, to about 2^-22 relative; results below 2^-126 are zero
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
// Registers per thread of a warpgroup, all of whose warps execute it.
template <int N>
__device__ __forceinline__ void set_regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

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
