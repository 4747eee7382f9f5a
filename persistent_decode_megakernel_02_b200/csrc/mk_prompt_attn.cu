// mk_prompt_attn.cu -- causal attention over packed prompts with grouped
// heads, on the tcgen05 tensor cores.
//
// Work is cut into units of (128 query rows of a sequence, query head); a
// block takes two units of one KV head, in the order (row block, head of the
// group), so that both share the K and V tiles they stream (128 keys each).
// A unit at row block b needs key tiles 0..b, the last one masked along its
// diagonal (row blocks and key tiles both start at the sequence's start).
//
// Per unit and key tile j:
//   S = Q K_j^T          (tcgen05, fp32 in tensor memory, M = N = 128)
//   P = exp2(c S - c m)  (one thread per row; m a running reference maximum)
//   O += P V_j           (P as 16-bit operand from tensor memory)
// The reference m is raised, and O rescaled, only when a tile's maximum
// exceeds it by more than 8 in the exponent of two: until then P stays
// below 2^8, which costs no precision, and the rescaling pass over O is
// rare.  l, the row's sum, stays in 32 bits in its thread; out = O / l.
//
// Roles: warps 0-3 and 4-7 the softmax of unit 0 and 1 (warp w reads tensor
// memory lanes 32 (w % 4)..), warp 8 a TMA loader (one thread), warp 9 the
// MMA issuer (one thread), warps 10-11 the guard of the masked tiles: a zero
// weight times a NaN or an infinity is not zero, so in the tiles that hold
// keys some row must not see, values that are not finite are taken out of
// shared memory and remembered per column with their first key; the epilogue
// adds them to the rows that do see them.
//
// Tensor memory: S0 | S1 | O0 | O1 (P overwrites the first half of its S).
#include <cuda.h>

#include <atomic>

#include "mk_tc.cuh"

namespace mk {
namespace {

constexpr int kTile = 128;                 // query rows of a unit, keys of a tile
constexpr int kPromptThreads = 384;
constexpr float kRescale = 8.f;            // exponent headroom before O is rescaled

template <int D>
struct PromptSmem {
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kStages = D == 64 ? 8 : 4;   // K and V tiles in flight
    static constexpr int kQ = 0;
    static constexpr int kRing = 2 * kTileBytes;
    static constexpr int kTail = kRing + kStages * kTileBytes;
    static constexpr int kBytes = kTail + 2560 + 1024;   // barriers, poison; slack to align the base
};

struct PromptTail {
    uint64_t q_full, full[8], empty[8], s_full[2], p_ready[2], o_full[2], guard_go[2], guard_done[2];
    uint32_t tmem;
    int abort;
    int any;             // a value was taken out
    int first[3][128];   // per column: first key (of the sequence) with NaN, +inf, -inf
};
static_assert(sizeof(PromptTail) <= 2560, "tail of the shared memory");

struct PromptParams {
    CUtensorMap q, k, v;
    PromptArgs a;
};

template <class T, int D>
__global__ void __launch_bounds__(kPromptThreads, 1) prompt_attn_kernel(const __grid_constant__ PromptParams p) {
    using L = PromptSmem<D>;
    constexpr bool kBf16 = T::kBf16;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = (unsigned char *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    PromptTail &t = *reinterpret_cast<PromptTail *>(smem + L::kTail);
    const PromptArgs &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.nq / a.nkv;

    // ---- the block's work: item `it` of a sequence, for KV head kvh
    if (blockIdx.x == 0)
        for (int i = tid; i < a.n_seqs; i += kPromptThreads) {
            const int b = a.cu[i], e = a.cu[i + 1];
            if (b < 0 || e < b || e > a.n_tokens || e - b > a.max_len) bad_value(a.status);
        }
    const int kvh = blockIdx.x % a.nkv;
    int it = blockIdx.x / a.nkv;
    int row0 = 0, len = 0, items = 0;
    for (int s0 = 0; s0 < a.n_seqs && items == 0; s0 += 32) {
        int b = 0, n = 0;
        if (s0 + lane < a.n_seqs) {
            b = a.cu[s0 + lane];
            const int e = a.cu[s0 + lane + 1];
            if (b >= 0 && e >= b && e <= a.n_tokens && e - b <= a.max_len) n = e - b;
        }
        const int mine = ((n + kTile - 1) / kTile * G + 1) / 2;
        int sum = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, sum > it);
        if (hit) {
            const int src = __ffs(hit) - 1;
            row0 = __shfl_sync(0xffffffffu, b, src);
            len = __shfl_sync(0xffffffffu, n, src);
            items = __shfl_sync(0xffffffffu, mine, src);
            it -= __shfl_sync(0xffffffffu, sum - mine, src);
        } else
            it -= __shfl_sync(0xffffffffu, sum, 31);
    }
    if (items == 0) return;
    it = items - 1 - it;   // the longest first
    const int units = (len + kTile - 1) / kTile * G;
    const int u0 = 2 * it;
    const bool two = u0 + 1 < units;
    const int blk0 = u0 / G, blk1 = two ? (u0 + 1) / G : blk0;
    const int head0 = kvh * G + u0 % G, head1 = two ? kvh * G + (u0 + 1) % G : head0;
    const int n0 = blk0 + 1, n1 = two ? blk1 + 1 : 0, J = two ? blk1 + 1 : n0;

    // ---- setup
    if (warp == 9) {
        if (lane == 0) {
            mbar_init(&t.q_full, 1);
            for (int i = 0; i < L::kStages; ++i) {
                mbar_init(&t.full[i], 1);
                mbar_init(&t.empty[i], 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(&t.s_full[i], 1);
                mbar_init(&t.p_ready[i], 4);
                mbar_init(&t.o_full[i], 1);
                mbar_init(&t.guard_go[i], 1);
                mbar_init(&t.guard_done[i], 2);
            }
            t.abort = 0;
            t.any = 0;
            fence_mbar_init();
        }
        __syncwarp();
        tmem_alloc(&t.tmem, 512);
    }
    if (warp < 8)
        for (int i = tid; i < 3 * 128; i += 256) t.first[i / 128][i % 128] = 0x7fffffff;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = t.tmem;

    if (warp == 8) {
        if (lane == 0) {
            // ---- loader: Q, then K0 V0 K1 V1 ...
            mbar_arrive_expect_tx(&t.q_full, (two ? 2 : 1) * L::kTileBytes);
            for (int h = 0; h < D / 64; ++h) {
                tma_load_3d(smem + L::kQ + h * kTile * 128, &p.q, h * 64, head0, row0 + blk0 * kTile, &t.q_full);
                if (two)
                    tma_load_3d(smem + L::kQ + L::kTileBytes + h * kTile * 128, &p.q, h * 64, head1,
                                row0 + blk1 * kTile, &t.q_full);
            }
            bool ok = true;
            for (int f = 0; f < 2 * J && ok; ++f) {
                const int st = f % L::kStages, use = f / L::kStages;
                if (use > 0) ok = mbar_wait(&t.empty[st], (use - 1) & 1, &t.abort);
                if (!ok) break;
                mbar_arrive_expect_tx(&t.full[st], L::kTileBytes);
                for (int h = 0; h < D / 64; ++h)
                    tma_load_3d(smem + L::kRing + st * L::kTileBytes + h * kTile * 128, f & 1 ? &p.v : &p.k, h * 64,
                                kvh, row0 + (f >> 1) * kTile, &t.full[st]);
            }
            // every tile used: nothing is in flight when the block ends
            for (int st = 0; st < L::kStages && ok; ++st) {
                const int uses = (2 * J - st + L::kStages - 1) / L::kStages;
                if (uses > 0) ok = mbar_wait(&t.empty[st], (uses - 1) & 1, &t.abort);
            }
        }
    } else if (warp == 9) {
        if (lane == 0) {
            // ---- MMA issuer
            const uint32_t ring = smem_addr(smem + L::kRing), qs = smem_addr(smem + L::kQ);
            constexpr uint32_t kIdS = f16_idesc(kBf16, false, kTile, kTile);
            constexpr uint32_t kIdO = f16_idesc(kBf16, true, kTile, D);
            auto qk = [&](int u, int f) {
                const uint32_t kb = ring + f % L::kStages * L::kTileBytes, qb = qs + u * L::kTileBytes;
                #pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint32_t off = (s >> 2) * kTile * 128 + (s & 3) * 32;
                    mma_ss(tmem + u * kTile, desc_sw128(qb + off, 16, 1024), desc_sw128(kb + off, 16, 1024), kIdS,
                           s > 0);
                }
                tc_commit(&t.s_full[u]);
            };
            auto pv = [&](int u, int f, bool first) {
                const uint32_t vb = ring + f % L::kStages * L::kTileBytes;
                for (int s = 0; s < kTile / 16; ++s)
                    mma_ts(tmem + 2 * kTile + u * D, tmem + u * kTile + s * 8,
                           desc_sw128(vb + s * 16 * 128, kTile * 128, 1024), kIdO, !first || s > 0);
            };
            auto full = [&](int f) { return mbar_wait(&t.full[f % L::kStages], (f / L::kStages) & 1, &t.abort); };
            bool ok = mbar_wait(&t.q_full, 0, &t.abort) && full(0);
            if (ok) {
                qk(0, 0);
                if (two) qk(1, 0);
                tc_commit(&t.empty[0]);
            }
            for (int j = 0; j < J && ok; ++j) {
                const int fv = 2 * j + 1, fk = 2 * j + 2;
                ok = full(fv);
                if (!ok) break;
                if (j >= blk0) mbar_arrive(&t.guard_go[j - blk0]);   // a masked tile (the last, or last two)
                for (int u = 0; u < 2 && ok; ++u) {
                    const int n = u ? n1 : n0;
                    if (j >= n) continue;
                    ok = mbar_wait(&t.p_ready[u], j & 1, &t.abort);
                    if (!ok) break;
                    if (j >= blk0) ok = mbar_wait(&t.guard_done[j - blk0], 0, &t.abort);
                    if (!ok) break;
                    tc_fence_after();
                    pv(u, fv, j == 0);
                    if (j + 1 < n) {
                        ok = full(fk);
                        if (ok) qk(u, fk);
                    } else
                        tc_commit(&t.o_full[u]);
                }
                if (!ok) break;
                tc_commit(&t.empty[fv % L::kStages]);
                if (j + 1 < J) tc_commit(&t.empty[fk % L::kStages]);
            }
        }
    } else if (warp >= 10) {
        // ---- guard of the masked tiles
        const int gt = tid - 10 * 32;
        bool ok = true;
        for (int which = 0; which < (blk1 != blk0 ? 2 : 1) && ok; ++which) {
            // the issuer says when the tile is there: a wait on the tile's own
            // barrier from here could miss phases of the tiles before it
            const int j = blk0 + which, f = 2 * j + 1;
            ok = mbar_wait_warp(&t.guard_go[which], 0, &t.abort) &&
                 mbar_wait_warp(&t.full[f % L::kStages], (f / L::kStages) & 1, &t.abort);
            if (!ok) break;
            uint4 *tile = reinterpret_cast<uint4 *>(smem + L::kRing + f % L::kStages * L::kTileBytes);
            constexpr uint32_t kExp = kBf16 ? 0x7f807f80u : 0x7c007c00u, kOne = kBf16 ? 0x00800080u : 0x04000400u;
            uint32_t bad = 0;
#pragma unroll 8
            for (int i = gt; i < L::kTileBytes / 16; i += 64) {
                const uint4 x = tile[i];
                bad |= ((x.x & kExp) + kOne) | ((x.y & kExp) + kOne) | ((x.z & kExp) + kOne) | ((x.w & kExp) + kOne);
            }
            if (bad & 0x80008000u) {
                uint16_t *e = reinterpret_cast<uint16_t *>(tile);
                for (int i = gt; i < L::kTileBytes / 16; i += 64)
                    for (int c = 0; c < 8; ++c) {
                        const uint32_t w = e[i * 8 + c];
                        if ((w & kExp & 0xffffu) != (kExp & 0xffffu)) continue;
                        e[i * 8 + c] = 0;
                        const int half = i / (kTile * 8), r = i / 8 % kTile;
                        const int col = half * 64 + ((i ^ r) & 7) * 8 + c;
                        if (j * kTile + r < len) {
                            const int kind = (w & ~kExp & 0x7fffu) ? 0 : w & 0x8000u ? 2 : 1;
                            atomicMin(&t.first[kind][col], j * kTile + r);
                            t.any = 1;
                        }
                    }
                fence_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&t.guard_done[which]);
        }
    } else {
        // ---- softmax: one row per thread
        const int u = warp >> 2, r = tid & 127;
        const int n = u ? n1 : n0, blk = u ? blk1 : blk0, head = u ? head1 : head0;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // lane 32 (w % 4) in bits 16..
        const uint32_t ts = tmem + u * kTile + lanes, to = tmem + 2 * kTile + u * D + lanes;
        const float c = a.scale * 1.4426950408889634f;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int j = 0; j < n && ok; ++j) {
            // S of this tile; the products of the tile before are done too (one
            // thread issues all of them, in this order)
            ok = mbar_wait_warp(&t.s_full[u], j & 1, &t.abort);
            if (!ok) break;
            tc_fence_after();
            const int limit = j == blk ? r : kTile;   // keys beyond it are not seen
            float top = -INFINITY;
            uint32_t x[32];
            for (int q = 0; q < 4; ++q) {
                tmem_ld32(ts + q * 32, x);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (q * 32 + i <= limit) top = fmaxf(top, __uint_as_float(x[i]));
            }
            const float old = m;
            if (!((top - m) * c <= kRescale)) m = fmaxf(m, top);
            const bool raise = m != old;
            if (__any_sync(0xffffffffu, raise)) {
                const float f = raise ? exp2f((old - m) * c) : 1.f;
                l *= f;
                if (j > 0) {
                    for (int q = 0; q < D / 32; ++q) {
                        tmem_ld32(to + q * 32, x);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
                        tmem_st32(to + q * 32, x);
                    }
                }
            }
            const float mc = m == -INFINITY ? 0.f : m * c;
            float sum = 0.f;
            for (int q = 0; q < 4; ++q) {
                tmem_ld32(ts + q * 32, x);
                tmem_ld_wait();
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    float e0 = exp2f(fmaf(__uint_as_float(x[i]), c, -mc));
                    float e1 = exp2f(fmaf(__uint_as_float(x[i + 1]), c, -mc));
                    if (q * 32 + i > limit) e0 = 0.f;
                    if (q * 32 + i + 1 > limit) e1 = 0.f;
                    sum += e0 + e1;
                    w[i / 2] = T::pack(e0, e1);
                }
                // columns 16 q.. of P: behind what this row has read of S
                tmem_st16(ts + q * 16, w);
            }
            l += sum;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&t.p_ready[u]);
        }
        if (ok && n > 0) ok = mbar_wait_warp(&t.o_full[u], 0, &t.abort);
        if (ok && n > 0) {
            tc_fence_after();
            const int pos = blk * kTile + r;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            uint16_t *dst = (uint16_t *)a.out + (long long)(row0 + pos) * a.out_stride + (long long)head * D;
            const bool any = t.any != 0;
            for (int q = 0; q < D / 32; ++q) {
                uint32_t x[32];
                tmem_ld32(to + q * 32, x);
                tmem_ld_wait();
                if (any)
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int col = q * 32 + i;
                        float o = __uint_as_float(x[i]);
                        if (t.first[0][col] <= pos) o = NAN;
                        if (t.first[1][col] <= pos) o += INFINITY;
                        if (t.first[2][col] <= pos) o -= INFINITY;
                        x[i] = __float_as_uint(o);
                    }
                if (pos < len)
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint4 w;
                        w.x = T::pack(__uint_as_float(x[i]) * inv, __uint_as_float(x[i + 1]) * inv);
                        w.y = T::pack(__uint_as_float(x[i + 2]) * inv, __uint_as_float(x[i + 3]) * inv);
                        w.z = T::pack(__uint_as_float(x[i + 4]) * inv, __uint_as_float(x[i + 5]) * inv);
                        w.w = T::pack(__uint_as_float(x[i + 6]) * inv, __uint_as_float(x[i + 7]) * inv);
                        *reinterpret_cast<uint4 *>(dst + q * 32 + i) = w;
                    }
            }
        }
    }

    // ---- teardown
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (t.abort) {
        // a wait ran out: say so, and let copies in flight land before the
        // shared memory is given up
        if (tid == 0 && a.status) *a.status = MK_ERR_TIMEOUT;
        const unsigned long long t0 = globaltimer();
        while (globaltimer() - t0 < 1000000ull) {}
    }
    if (warp == 9) tmem_dealloc(tmem, 512);
}

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static std::atomic<void *> fn{nullptr};
    void *f = fn.load(std::memory_order_relaxed);
    if (!f) {
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) !=
                cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(f, std::memory_order_relaxed);
    }
    return (EncodeFn)f;
}

// Map of a [tokens][heads][d] buffer: boxes of 64 elements of one head for
// 128 tokens, in the 128-byte swizzle; rows beyond the buffer read as zero.
bool make_map(CUtensorMap *m, int dtype, const void *ptr, int d, int heads, long long tokens, long long stride) {
    EncodeFn f = encode_fn();
    if (!f) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, kTile}, ones[3] = {1, 1, 1};
    return f(m, dtype == MK_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
             const_cast<void *>(ptr), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, int D>
cudaError_t launch(const PromptParams &p, int device, int grid, cudaStream_t stream) {
    static std::atomic<bool> ready[kOpsMaxDevices];
    if (!ready[device].load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute(prompt_attn_kernel<T, D>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, PromptSmem<D>::kBytes);
        if (e != cudaSuccess) return e;
        ready[device].store(true, std::memory_order_relaxed);
    }
    prompt_attn_kernel<T, D><<<grid, kPromptThreads, PromptSmem<D>::kBytes, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t prompt_launch(const PromptArgs &a, int device, int, cudaStream_t stream) {
    PromptParams p;
    p.a = a;
    if (!make_map(&p.q, a.dtype, a.q, a.d, a.nq, a.n_tokens, a.q_stride) ||
        !make_map(&p.k, a.dtype, a.k, a.d, a.nkv, a.n_tokens, a.k_stride) ||
        !make_map(&p.v, a.dtype, a.v, a.d, a.nkv, a.n_tokens, a.v_stride))
        return cudaErrorInvalidValue;
    // at most this many items: a sequence of n row blocks has ceil(n G / 2) per KV head
    const long long G = a.nq / a.nkv, top = a.max_len < a.n_tokens ? a.max_len : a.n_tokens;
    long long blocks = a.n_tokens / kTile + a.n_seqs;
    const long long most = a.n_seqs * ((top + kTile - 1) / kTile);
    if (most < blocks) blocks = most;
    long long grid = (blocks * G + a.n_seqs + 1) / 2 * a.nkv;
    if (grid < 1) grid = 1;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (a.dtype == MK_BF16)
        return a.d == 64 ? launch<Bf16, 64>(p, device, (int)grid, stream)
                         : launch<Bf16, 128>(p, device, (int)grid, stream);
    return a.d == 64 ? launch<Fp16, 64>(p, device, (int)grid, stream)
                     : launch<Fp16, 128>(p, device, (int)grid, stream);
}

}  // namespace mk
