// mk_tc.cuh -- TMA tile loads, swizzled shared-memory descriptors and
// tcgen05.mma forms of the prompt attention kernel, and its bounded barrier
// waits.  Device code only; not part of the public ABI.
#pragma once

#include <cuda.h>   // CUtensorMap

#include "mk_ops.cuh"

namespace mk {

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Shared-memory matrix descriptor with the 128-byte swizzle (rows of 128
// bytes, groups of 8 rows 1024 bytes apart).  For a K-major operand the
// stride offset is that of the 8-row groups; for an MN-major one (rows run
// along K) it is that of 8 K-rows, and the leading offset separates blocks of
// 64 elements along MN.
// `at` is the shared-memory address / 16; the high word is a constant.
__device__ __forceinline__ uint64_t desc_sw128_at(uint32_t at, uint32_t lbo, uint32_t sbo) {
    return ((uint64_t)((sbo >> 4) | 1u << 14 | 2u << 29) << 32) | (at | (lbo >> 4) << 16);
}
// One thread of the warp (all 32 lanes call it).
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}
// Instruction descriptor of kind::f16: fp32 accumulator, both operands bf16
// (or both fp16), A K-major, B K-major or MN-major.
__host__ __device__ constexpr uint32_t f16_idesc(bool bf16, bool b_mn, int m, int n) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
// D += A B (acc = 0: D = A B); A from shared memory
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// the same with A from tensor memory
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// 16 consecutive 32-bit columns of this thread's lane (warp-wide)
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(
            r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void fence_mbar_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// Wait for a barrier's phase, bounded: after kWaitTries tries, each of which
// may itself wait a while (seconds in all), or once another role of the block
// has given up, it returns false with *abort set.  Kept to a few instructions:
// it is inlined at every wait.
constexpr uint32_t kWaitTries = 1u << 23;
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    uint32_t tries = 0;
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
        if ((++tries & 255u) == 0 && (tries >= kWaitTries || *abort)) {
            *abort = 1;
            return false;
        }
    }
    return true;
}
// the same for a whole warp, with one answer
__device__ __forceinline__ bool mbar_wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}

}  // namespace mk
