// mk_prompt_attn.cu -- causal attention over packed prompts with grouped
// heads, on the tcgen05 tensor cores.
//
// Work is cut into units of (128 query rows of a sequence, query head); an
// item is two units of one KV head that share the K and V tiles they stream
// (128 keys each): two heads of a row block, or, where the group is odd,
// neighbours in the order (row block, head) of two row blocks.  A unit at row
// block b needs key tiles 0..b, the last one masked along its diagonal (row
// blocks and key tiles both start at the sequence's start).  One block per SM
// walks the items, longest first over all sequences, in a there-and-back
// order (block c takes c, 2P - 1 - c, 2P + c, ...), which needs no counter and
// leaves the blocks' sums close; the next item's loads and first products
// start while the last one's outputs are written.
//
// Per unit and key tile j:
//   S = Q K_j^T          (tcgen05, fp32 in tensor memory, M = N = 128)
//   P = exp2(c S - c m)  (one thread per row; m a running reference maximum)
//   O += P V_j           (P as 16-bit operand from tensor memory)
// The reference m is raised, and O rescaled, only when a tile's maximum
// exceeds it by more than 8 (fp16: 4) in the exponent of two: until then P stays
// below a power of two that costs no precision, and the rescaling pass over O
// is rare.  l, the row's sum, stays in 32 bits in its thread; out = O / l.
//
// Roles: warps 0-3 and 4-7 the softmax of unit 0 and 1 (warp w reads tensor
// memory lanes 32 (w % 4)..), warp 8 the scheduler and TMA loader, warp 9 the
// MMA issuer, warps 10-11 the guard of the masked tiles: a zero
// weight times a NaN or an infinity is not zero, so in the tiles that hold
// keys some row must not see, values that are not finite are taken out of
// shared memory and remembered per column with their first key; the epilogue
// adds them to the rows that do see them.  Each guard warp has half of the
// columns to itself, so that the two never wait for one another.
//
// The code is kept small (loops over sequences, a tile's loads and the rare
// paths are not unrolled): at 92 KB the SMs fetched most of every short item's
// code from the instruction cache that a cluster of them shares, at 92 % of
// its rate.  At 66 KB 1000 prompts of 20 tokens took 524 us instead of 559 (532
// since the guard's warps have their own columns), 100 of 200 tokens 130 instead
// of 142; rolling the epilogue and the issuer's loop
// over the units too (53 KB) gives 469 and 135, but costs long prompts 5 %.
//
// What bounds it: a unit's tile is a chain (products, softmax, products; 1024
// cycles of matrix work at 128 dims, and 1320 of a softmax warp alone, 1760
// beside the other unit's), of which the two units overlap two: 8192 tokens
// of 32/8/128 heads 442 us, 1.24 PFLOP/s, 77 % of the matrix peak measured in
// bursts.  With 64 dims the products are half of that and the chain's latency
// remains: 6811 tokens in 9 prompts 73 us, with the matrix unit 22 %, the unit of
// the exponentials 51 % and the issue slots 37 % busy -- two units in flight and two
// softmax warps a scheduler do not fill any of them.  Short prompts by the
// latency of one tile's chain from load to store.
//
// Tensor memory, 512 columns: S0 | S1 | O0 | O1, and for 64 dims P0 | P1: the
// next tile's S is then computed while this one's softmax runs.  For 128 dims
// P lies over the first half of its S.
#include <cuda.h>

#include <atomic>

#include "mk_tc.cuh"

namespace mk {
namespace {

constexpr int kTile = 128;                 // query rows of a unit, keys of a tile
constexpr int kPromptThreads = 384;
// Registers: launched at 168 a thread (65536 / 384, rounded down to 8), moved
// from the control warpgroup to the softmax ones, whose row of S stays in
// registers.  The shares must add up to the launch's, or the wait for more
// registers would not end: prompt_launch refuses any other launch count.
constexpr int kLaunchRegsPrompt = 168, kSoftmaxRegs = 208, kControlRegsPrompt = 88;
static_assert(256 * kSoftmaxRegs + 128 * kControlRegsPrompt == kPromptThreads * kLaunchRegsPrompt, "register split");
// Exponent headroom before O is rescaled, and the scale of the weights, P =
// 2^(score - reference + kScale).  fp16 has no exponents to spare: P goes up to
// 2^15, so that a weight keeps its 11 bits down to 2^-25 of the row's largest and
// is off by at most 2^-36 of it below.  (Headroom 8 / 4 / 2 / 0 in fp16: 8192 tokens
// of 32/8/128 heads 463, 462, 498, 515 us with scores of N(0, 1), 477, 504, 510, 515
// with three times their spread; unscaled 461 and 476, and weights of 2^-20 of the
// largest off by 3 %, gone below 2^-25.)
template <class T>
struct PromptWeight {
    static constexpr float kRescale = T::kBf16 ? 8.f : 4.f, kScale = T::kBf16 ? 0.f : 11.f;
};

// The larger of three (NaN is left out, as by fmaxf).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <int D>
struct PromptSmem {
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kStages = D == 64 ? 8 : 4;   // K and V tiles in flight
    static constexpr int kQ = 0;
    static constexpr int kRing = 2 * kTileBytes;
    static constexpr int kTail = kRing + kStages * kTileBytes;
    static constexpr int kStore = kTail + 4096;          // 2 KB a softmax warp: 32 rows of 32 output columns
    static constexpr int kBytes = kStore + 8 * 2048;
};

struct PromptItem {
    int row0, len;                 // the sequence's first row and length; len 0: no more items
    int tiles;                     // key tiles of the longer unit
    int blk[2], head[2], n[2];     // per unit: row block, query head, key tiles (0: no such unit)
};

// Every barrier's phases run on from item to item.
struct PromptTail {
    uint64_t full[8], empty[8];               // the ring of K and V tiles
    uint64_t q_full, q_empty;                 // both units' queries
    uint64_t s_full[2], s_free[2], p_ready[2], pv_done[2];   // per tile
    uint64_t o_full[2], o_empty[2];           // per item
    uint64_t guard_go[2], guard_done[2];      // the first and second masked tile of an item
    uint64_t item_full[2], item_empty[2];
    PromptItem item[2];
    uint32_t tmem;
    int abort;
    int any[2][2];          // a value was taken out, by the guard warp of its column
    int first[2][3][128];   // per column: first key (of the sequence) with NaN, +inf, -inf
};
static_assert(sizeof(PromptTail) <= 4096, "tail of the shared memory");

struct PromptParams {
    CUtensorMap q, k, v;
    PromptArgs a;
};

template <class T, int D>
__global__ void __launch_bounds__(kPromptThreads, 1) prompt_attn_kernel(const __grid_constant__ PromptParams p) {
    using L = PromptSmem<D>;
    using W = PromptWeight<T>;
    constexpr bool kBf16 = T::kBf16;
    extern __shared__ __align__(1024) unsigned char smem[];
    PromptTail &t = *reinterpret_cast<PromptTail *>(smem + L::kTail);
    const PromptArgs &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (smem_addr(smem) & 1023u) {      // the swizzled tiles need it; no static shared memory comes before
        if (tid == 0) bad_value(a.status);
        return;
    }

    if (blockIdx.x == 0)
#pragma unroll 1
        for (int i = tid; i < a.n_seqs; i += kPromptThreads) {
            const int b = a.cu[i], e = a.cu[i + 1];
            if (b < 0 || e < b || e > a.n_tokens || e - b > a.max_len) bad_value(a.status);
        }

    // ---- setup
    if (warp == 9) {
        if (lane == 0) {
            for (int i = 0; i < L::kStages; ++i) {
                mbar_init(&t.full[i], 1);
                mbar_init(&t.empty[i], 1);
            }
            mbar_init(&t.q_full, 1);
            mbar_init(&t.q_empty, 1);
            for (int i = 0; i < 2; ++i) {
                mbar_init(&t.s_full[i], 1);
                mbar_init(&t.s_free[i], 4);
                mbar_init(&t.p_ready[i], 4);
                mbar_init(&t.pv_done[i], 1);
                mbar_init(&t.o_full[i], 1);
                mbar_init(&t.o_empty[i], 4);
                mbar_init(&t.guard_go[i], 1);
                mbar_init(&t.guard_done[i], 2);
                mbar_init(&t.item_full[i], 1);
                mbar_init(&t.item_empty[i], 11);   // issuer, 2 guard and 8 softmax warps
                t.any[i][0] = t.any[i][1] = 0;
            }
            t.abort = 0;
            fence_mbar_init();
        }
        __syncwarp();
        tmem_alloc(&t.tmem, 512);
    }
    if (warp < 8)
        for (int i = tid; i < 2 * 3 * 128; i += 256) (&t.first[0][0][0])[i] = 0x7fffffff;
    // the loader's view of the work, begun while the others set up: level l of
    // a sequence is its row blocks R l .. R l + R - 1
    const int G = a.nq / a.nkv, R = G & 1 ? 2 : 1;
    const int per_seq = G * R / 2 * a.nkv;            // items of a sequence at a level
    int row0 = 0, len = 0;      // of sequence s0 + lane
    auto levels_of = [&](int s) {
        row0 = len = 0;
        if (s < a.n_seqs) {
            const int b = a.cu[s], e = a.cu[s + 1];
            if (b >= 0 && e >= b && e <= a.n_tokens && e - b <= a.max_len) {
                row0 = b;
                len = e - b;
            }
        }
        return (len + kTile * R - 1) / (kTile * R);
    };
    // sequences that have a level; down to level `low` they are the same, so
    // the lengths are read once per different number of levels
    int low = 0;
    auto count = [&](int level) {
        int c = 0, shorter = 0;
#pragma unroll 1
        for (int s0 = 0; s0 < a.n_seqs; s0 += 32) {
            const int levels = levels_of(s0 + lane);
            c += __popc(__ballot_sync(0xffffffffu, levels > level));
            if (levels <= level) shorter = max(shorter, levels);
        }
        low = __reduce_max_sync(0xffffffffu, shorter);
        return c;
    };
    int level = 0;
    if (warp == 8) {
        if (lane < 3) tma_prefetch_map(lane == 0 ? &p.q : lane == 1 ? &p.k : &p.v);
#pragma unroll 1
        for (int s0 = 0; s0 < a.n_seqs; s0 += 32) level = max(level, levels_of(s0 + lane));
        low = level = __reduce_max_sync(0xffffffffu, level);      // above the highest
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, t.tmem, 0);

    if (warp >= 8) set_regs_down<kControlRegsPrompt>();
    if (warp == 8) {
        // ---- scheduler and loader
        uint32_t base = 0;           // items before the level
        int here = 0;                // sequences that have it
        int at = 0, passed = 0;      // those before sequence `at`: the search goes on from there
        const uint32_t P = gridDim.x;
        int k = 0, F = 0;     // items published, tiles loaded
        bool ok = true;
        for (uint32_t turn = 0; ok; ++turn) {
            const uint32_t rank = turn * P + (turn & 1 ? P - 1 - blockIdx.x : blockIdx.x);
            while (level >= 0 && rank >= base + (uint32_t)here * per_seq) {
                base += (uint32_t)here * per_seq;
                --level;
                at = passed = 0;
                if (level < low) here = level >= 0 ? count(level) : 0;
            }
            // lanes 0 and 1 hold a unit each
            int seq_row = 0, seq_len = 0, kvh = 0, head = 0, blk = 0, n = 0;
            if (level >= 0) {
                const int nth = (int)((rank - base) / per_seq), rem = (int)(rank - base - (uint32_t)nth * per_seq);
#pragma unroll 1
                for (; at < a.n_seqs; at += 32) {
                    const unsigned m = __ballot_sync(0xffffffffu, levels_of(at + lane) > level);
                    const int ahead = nth - passed;
                    if (ahead < __popc(m)) {
                        const bool me = (m >> lane & 1u) && __popc(m & ((1u << lane) - 1)) == ahead;
                        const int src = __ffs(__ballot_sync(0xffffffffu, me)) - 1;
                        seq_row = __shfl_sync(0xffffffffu, row0, src);
                        seq_len = __shfl_sync(0xffffffffu, len, src);
                        break;
                    }
                    passed += __popc(m);
                }
                const int pair = rem / a.nkv, unit = pair * 2 + (lane & 1), row_blk = unit / G;
                kvh = rem - pair * a.nkv;
                head = kvh * G + unit - row_blk * G;
                blk = level * R + row_blk;
                if (blk < (seq_len + kTile - 1) / kTile) n = blk + 1;
            }
            const int n0 = __shfl_sync(0xffffffffu, n, 0), n1 = __shfl_sync(0xffffffffu, n, 1), tiles = max(n0, n1);
            if (level >= 0 && n0 == 0) continue;      // a lone last row block has half the units
            const int slot = k & 1;
            if (k >= 2) ok = mbar_wait_warp(&t.item_empty[slot], ((k >> 1) - 1) & 1, &t.abort);
            if (!ok) break;
            PromptItem &it = t.item[slot];
            const int blk0 = __shfl_sync(0xffffffffu, blk, 0);
            if (lane < 2) {
                it.head[lane] = head;
                it.blk[lane] = n ? blk : blk0;
                it.n[lane] = n;
            }
            if (lane == 0) {
                it.row0 = seq_row;
                it.len = seq_len;
                it.tiles = tiles;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&t.item_full[slot]);
            if (level < 0) break;
            if (k > 0) ok = mbar_wait_warp(&t.q_empty, (k - 1) & 1, &t.abort);
            if (!ok) break;
            ++k;
            const int units = n1 ? 2 : 1;
            if (lane == 0) mbar_arrive_expect_tx(&t.q_full, units * L::kTileBytes);
            __syncwarp();
            if (lane < units)
                for (int h = 0; h < D / 64; ++h)
                    tma_load_3d(smem + L::kQ + lane * L::kTileBytes + h * kTile * 128, &p.q, h * 64, head, seq_row + blk * kTile,
                                &t.q_full);
#pragma unroll 1
            for (int f = 0; f < 2 * tiles && ok; ++f, ++F) {       // K0 V0 K1 V1 ...
                const int st = F % L::kStages, use = F / L::kStages;
                if (use > 0) ok = mbar_wait_warp(&t.empty[st], (use - 1) & 1, &t.abort);
                if (ok && lane == 0) {
                    mbar_arrive_expect_tx(&t.full[st], L::kTileBytes);
                    for (int h = 0; h < D / 64; ++h)
                        tma_load_3d(smem + L::kRing + st * L::kTileBytes + h * kTile * 128, f & 1 ? &p.v : &p.k, h * 64,
                                    kvh, seq_row + (f >> 1) * kTile, &t.full[st]);
                }
            }
        }
        // every tile used: nothing is in flight when the block ends
#pragma unroll 1
        for (int st = 0; st < L::kStages && ok; ++st) {
            const int uses = (F - st + L::kStages - 1) / L::kStages;
            if (uses > 0) ok = mbar_wait_warp(&t.empty[st], (uses - 1) & 1, &t.abort);
        }
    } else if (warp == 9) {
        // ---- MMA issuer: the whole warp walks the loop (addresses stay
        // uniform), one elected thread issues.  With a single thread walking
        // it, every operand went through a vector register first: 78 cycles
        // an instruction instead of the 64 it computes.
        const bool leader = elect_one();
        const uint32_t ring = (smem_addr(smem + L::kRing) & 0x3FFFFu) >> 4, qs = (smem_addr(smem + L::kQ) & 0x3FFFFu) >> 4;
        constexpr uint32_t kIdS = f16_idesc(kBf16, false, kTile, kTile);
        constexpr uint32_t kIdO = f16_idesc(kBf16, true, kTile, D);
        constexpr bool kOwnP = D == 64;
        auto qk = [&](int u, int f) {
            const uint32_t kb = ring + (f % L::kStages) * (L::kTileBytes >> 4), qb = qs + u * (L::kTileBytes >> 4);
            if (leader) {
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint32_t off = ((s >> 2) * kTile * 128 + (s & 3) * 32) >> 4;
                    mma_ss(tmem + u * kTile, desc_sw128_at(qb + off, 16, 1024), desc_sw128_at(kb + off, 16, 1024), kIdS,
                           s > 0);
                }
                tc_commit(&t.s_full[u]);
            }
        };
        auto pv = [&](int u, int f, bool first, bool last) {
            const uint32_t vb = ring + (f % L::kStages) * (L::kTileBytes >> 4);
            const uint32_t pb = tmem + (kOwnP ? 2 * kTile + 2 * D + u * 64 : u * kTile);
            if (leader) {
#pragma unroll
                for (int s = 0; s < kTile / 16; ++s)
                    mma_ts(tmem + 2 * kTile + u * D, pb + s * 8,
                           desc_sw128_at(vb + (s * 16 * 128 >> 4), kTile * 128, 1024), kIdO, s > 0 || !first);
                if (kOwnP) tc_commit(&t.pv_done[u]);
                if (last) tc_commit(&t.o_full[u]);
            }
        };
        auto full = [&](int f) {
            return mbar_wait_warp(&t.full[f % L::kStages], (f / L::kStages) & 1, &t.abort);
        };
        int F = 0, products[2] = {0, 0}, tiles[2] = {0, 0}, outs[2] = {0, 0}, masked[2] = {0, 0};    // phases so far
        bool ok = true;
        for (int k = 0; ok; ++k) {
            ok = mbar_wait_warp(&t.item_full[k & 1], (k >> 1) & 1, &t.abort);
            if (!ok) break;
            const PromptItem &it = t.item[k & 1];
            const int J = __shfl_sync(0xffffffffu, it.tiles, 0), blk0 = __shfl_sync(0xffffffffu, it.blk[0], 0);
            const int n0 = __shfl_sync(0xffffffffu, it.n[0], 0), n1 = __shfl_sync(0xffffffffu, it.n[1], 0);
            __syncwarp();
            if (J == 0) break;
            if (leader) mbar_arrive(&t.item_empty[k & 1]);
            ok = mbar_wait_warp(&t.q_full, k & 1, &t.abort);
            // S of the units that have tile j
            auto both_qk = [&](int j) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (j >= (u ? n1 : n0) || !ok) continue;
                    if (kOwnP) {
                        // (of a fresh barrier the phase before the first counts as over)
                        ok = mbar_wait_warp(&t.s_free[u], (products[u]++ & 1) ^ 1, &t.abort);
                        tc_fence_after();
                    }
                    if (ok) ok = full(F + 2 * j);
                    if (ok) qk(u, F + 2 * j);
                }
            };
            auto qk_used = [&](int j) {       // tile j's keys, and with the last one the queries
                if (!ok || !leader) return;
                tc_commit(&t.empty[(F + 2 * j) % L::kStages]);
                if (j + 1 == J) tc_commit(&t.q_empty);
            };
            if (ok) both_qk(0);
            qk_used(0);
            for (int j = 0; j < J && ok; ++j) {
                const int fv = F + 2 * j + 1;
                ok = full(fv);
                if (!ok) break;
                const bool mask = j >= blk0;      // the last tile, or the last two
                if (mask && leader) mbar_arrive(&t.guard_go[j - blk0]);
                if (kOwnP && j + 1 < J) {
                    both_qk(j + 1);
                    qk_used(j + 1);
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int n = u ? n1 : n0;
                    if (j >= n || !ok) continue;
                    ok = mbar_wait_warp(&t.p_ready[u], tiles[u]++ & 1, &t.abort);
                    if (ok && j == 0) ok = mbar_wait_warp(&t.o_empty[u], (outs[u] & 1) ^ 1, &t.abort);
                    if (ok && mask)
                        ok = mbar_wait_warp(&t.guard_done[j - blk0], (j == blk0 ? masked[0] : masked[1]) & 1, &t.abort);
                    if (!ok) continue;
                    tc_fence_after();
                    pv(u, fv, j == 0, j + 1 == n);
                    if (!kOwnP && j + 1 < n) {
                        ok = full(fv + 1);
                        if (ok) qk(u, fv + 1);
                    }
                }
                if (ok && leader) tc_commit(&t.empty[fv % L::kStages]);
                if (!kOwnP && j + 1 < J) qk_used(j + 1);
            }
            ++masked[0];
            if (J - 1 > blk0) ++masked[1];
            ++outs[0];
            if (n1) ++outs[1];
            F += 2 * J;
        }
    } else if (warp >= 10) {
        // ---- guard of the masked tiles
        const int half = warp - 10;
        int F = 0, masked[2] = {0, 0};
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const int slot = k & 1;
            ok = mbar_wait_warp(&t.item_full[slot], (k >> 1) & 1, &t.abort);
            if (!ok) break;
            const int J = t.item[slot].tiles, blk0 = t.item[slot].blk[0], len = t.item[slot].len;
            if (J == 0) break;
            if (t.any[slot][half]) {       // what the item before last left here
                __syncwarp();
                for (int i = lane; i < D / 2; i += 32)
                    for (int kind = 0; kind < 3; ++kind) t.first[slot][kind][half * (D / 2) + i] = 0x7fffffff;
                if (lane == 0) t.any[slot][half] = 0;
                __syncwarp();
            }
            for (int which = 0; which < J - blk0 && ok; ++which) {
                // the issuer says when the tile is there: a wait on the tile's own
                // barrier from here could miss phases of the tiles before it
                const int j = blk0 + which, f = F + 2 * j + 1;
                ok = mbar_wait_warp(&t.guard_go[which], masked[which]++ & 1, &t.abort) &&
                     mbar_wait_warp(&t.full[f % L::kStages], (f / L::kStages) & 1, &t.abort);
                if (!ok) break;
                uint4 *tile = reinterpret_cast<uint4 *>(smem + L::kRing + f % L::kStages * L::kTileBytes);
                constexpr int kSteps = L::kTileBytes / 16 / 64;
                constexpr uint32_t kExp = kBf16 ? 0x7f807f80u : 0x7c007c00u, kOne = kBf16 ? 0x00800080u : 0x04000400u;
                uint32_t bad = 0;
#pragma unroll 4
                for (int step = 0; step < kSteps; ++step) {
                    const uint4 x = tile[guard_vector(D, half, step, lane)];
                    bad |= ((x.x & kExp) + kOne) | ((x.y & kExp) + kOne) | ((x.z & kExp) + kOne) | ((x.w & kExp) + kOne);
                }
                if (bad & 0x80008000u) {
                    uint16_t *e = reinterpret_cast<uint16_t *>(tile);
#pragma unroll 1
                    for (int step = 0; step < kSteps; ++step) {
                        const int i = guard_vector(D, half, step, lane), r = guard_row(i);
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) {
                            const uint32_t w = e[i * 8 + c];
                            if ((w & kExp & 0xffffu) != (kExp & 0xffffu)) continue;
                            e[i * 8 + c] = 0;
                            const int col = guard_column(i) + c;
                            if (j * kTile + r < len) {
                                const int kind = (w & ~kExp & 0x7fffu) ? 0 : w & 0x8000u ? 2 : 1;
                                atomicMin(&t.first[slot][kind][col], j * kTile + r);
                                t.any[slot][half] = 1;
                            }
                        }
                    }
                    fence_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&t.guard_done[which]);
            }
            if (lane == 0) mbar_arrive(&t.item_empty[slot]);
            F += 2 * J;
        }
    } else {
        // ---- softmax: one row per thread
        set_regs_up<kSoftmaxRegs>();
        const int u = warp >> 2, r = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // lane 32 (w % 4) in bits 16..
        const uint32_t ts = tmem + u * kTile + lanes, to = tmem + 2 * kTile + u * D + lanes;
        constexpr bool kOwnP = D == 64;
        const uint32_t tp = kOwnP ? tmem + 2 * kTile + 2 * D + u * 64 + lanes : ts;
        const float c = a.scale * 1.4426950408889634f;
        int tiles = 0, outs = 0, pvs = 0;      // phases so far
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const int slot = k & 1;
            ok = mbar_wait_warp(&t.item_full[slot], (k >> 1) & 1, &t.abort);
            if (!ok || t.item[slot].tiles == 0) break;
            const int n = t.item[slot].n[u], blk = t.item[slot].blk[u];
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < n && ok; ++j) {
                // S of this tile (for 128 dims the products of the tile before are
                // done too: one thread issues all of them, in this order)
                ok = mbar_wait_warp(&t.s_full[u], tiles++ & 1, &t.abort);
                if (!ok) break;
                tc_fence_after();
                uint32_t x[4][32];
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_ld32(ts + q * 32, x[q]);
                tmem_ld_wait();
                if constexpr (kOwnP) {      // S is read: the next tile's may be computed
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&t.s_free[u]);
                }
                if (j == blk)      // the diagonal: keys beyond the row's own are not seen
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int n = r + 1 - q * 32;      // of these 32 are seen
                        const uint32_t hide = n <= 0 ? 0xffffffffu : n >= 32 ? 0u : 0xffffffffu << n;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (hide >> i & 1u) x[q][i] = 0xff800000u;
                    }
                auto at = [&](int i) { return __uint_as_float(x[i / 32][i % 32]); };
                float top4[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) top4[i] = max3(at(i), at(i + 4), at(i + 8));
#pragma unroll
                for (int i = 12; i < kTile - 4; i += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k) top4[k] = max3(top4[k], at(i + k), at(i + k + 4));
#pragma unroll
                for (int k = 0; k < 4; ++k) top4[k] = max3(top4[k], at(kTile - 4 + k), top4[k]);
                const float top = max3(max3(top4[0], top4[1], top4[2]), top4[3], top4[3]);
                const float old = m;
                if (!((top - m) * c <= W::kRescale)) m = fmaxf(m, top);
                const bool raise = m != old;
                // P and O are free once the tile before is weighted (128 dims: it is)
                auto weighted = [&] {
                    if (!kOwnP || j == 0) return true;
                    const bool done = mbar_wait_warp(&t.pv_done[u], pvs & 1, &t.abort);
                    tc_fence_after();
                    return done;
                };
                if (__any_sync(0xffffffffu, raise)) {
                    const float f = raise ? ex2((old - m) * c) : 1.f;
                    l *= f;
                    ok = weighted();
                    if (!ok) break;
                    if (j > 0)
#pragma unroll 1
                        for (int q = 0; q < D / 16; ++q) {
                            uint32_t o[16];
                            tmem_ld16(to + q * 16, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st16(to + q * 16, o);
                        }
                }
                const float mc = m == -INFINITY ? 0.f : m * c;
                const float2 c2 = make_float2(c, c), mc2 = make_float2(W::kScale - mc, W::kScale - mc);
                float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
                // (a share of the exponentials on the FMA units, by a polynomial,
                // changed nothing between none and a quarter: 460, 459, 462 us at
                // 8192 tokens)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        float2 e0 = ffma2(make_float2(at(q * 32 + i), at(q * 32 + i + 1)), c2, mc2);
                        float2 e1 = ffma2(make_float2(at(q * 32 + i + 2), at(q * 32 + i + 3)), c2, mc2);
                        e0.x = ex2(e0.x);
                        e0.y = ex2(e0.y);
                        e1.x = ex2(e1.x);
                        e1.y = ex2(e1.y);
                        sum0 = fadd2(sum0, e0);
                        sum1 = fadd2(sum1, e1);
                        w[i / 2] = T::pack(e0.x, e0.y);
                        w[i / 2 + 1] = T::pack(e1.x, e1.y);
                    }
                    if (q == 0) ok = weighted();
                    tmem_st16(tp + q * 16, w);      // (128 dims: over what this row has read of S)
                }
                if (!ok) break;
                if (kOwnP && j > 0) ++pvs;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&t.p_ready[u]);
                l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
            }
            if (kOwnP && ok && n > 0) ok = mbar_wait_warp(&t.pv_done[u], pvs++ & 1, &t.abort);
            if (ok && n > 0) ok = mbar_wait_warp(&t.o_full[u], outs++ & 1, &t.abort);
            if (ok && n > 0) {
                tc_fence_after();
                const int pos = blk * kTile + r, len = t.item[slot].len;
                const float inv = l == 0.f ? 0.f : 1.f / l;
                // rows leave through shared memory, eight rows of 64 bytes a store:
                // one row a thread took 32 transactions a store instruction (the
                // epilogue 7400 cycles at 128 dims)
                uint4 *stage = reinterpret_cast<uint4 *>(smem + L::kStore + warp * 2048);
                auto staged = [&](int row, int chunk) { return stage + row * 4 + (chunk ^ (row >> 1 & 3)); };
                const int row_first = blk * kTile + (warp & 3) * 32;
                uint16_t *dst = (uint16_t *)a.out + (long long)(t.item[slot].row0 + row_first) * a.out_stride +
                                (long long)t.item[slot].head[u] * D;
                const bool any = (t.any[slot][0] | t.any[slot][1]) != 0;
#pragma unroll
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t x[32];
                    tmem_ld32(to + q * 32, x);
                    tmem_ld_wait();
                    if (q == D / 32 - 1) {      // O is read: the next item may start its own
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&t.o_empty[u]);
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint4 w;
                        w.x = T::pack(__uint_as_float(x[i]) * inv, __uint_as_float(x[i + 1]) * inv);
                        w.y = T::pack(__uint_as_float(x[i + 2]) * inv, __uint_as_float(x[i + 3]) * inv);
                        w.z = T::pack(__uint_as_float(x[i + 4]) * inv, __uint_as_float(x[i + 5]) * inv);
                        w.w = T::pack(__uint_as_float(x[i + 6]) * inv, __uint_as_float(x[i + 7]) * inv);
                        *staged(lane, i / 8) = w;
                    }
                    if (any)
#pragma unroll 1
                        for (int i = 0; i < 32; ++i) {
                            const int col = q * 32 + i;
                            uint16_t *e = reinterpret_cast<uint16_t *>(staged(lane, i / 8)) + i % 8;
                            float o = T::unpack(*e).x;
                            if (t.first[slot][0][col] <= pos) o = NAN;
                            if (t.first[slot][1][col] <= pos) o += INFINITY;
                            if (t.first[slot][2][col] <= pos) o -= INFINITY;
                            *e = (uint16_t)T::pack(o, 0.f);
                        }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = i * 8 + (lane >> 2), chunk = lane & 3;
                        if (row_first + row < len)
                            *reinterpret_cast<uint4 *>(dst + row * a.out_stride + q * 32 + chunk * 8) = *staged(row, chunk);
                    }
                    __syncwarp();
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&t.item_empty[slot]);
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
        cudaFuncAttributes at;
        const cudaError_t f = cudaFuncGetAttributes(&at, prompt_attn_kernel<T, D>);
        if (f != cudaSuccess) return f;
        if (at.numRegs != kLaunchRegsPrompt) return cudaErrorInvalidDeviceFunction;
        ready[device].store(true, std::memory_order_relaxed);
    }
    return launch_kernel(prompt_attn_kernel<T, D>, grid, kPromptThreads, PromptSmem<D>::kBytes, stream, p);
}

}  // namespace

cudaError_t prompt_launch(const PromptArgs &a, int device, int num_sms, cudaStream_t stream) {
    PromptParams p;
    p.a = a;
    if (!make_map(&p.q, a.dtype, a.q, a.d, a.nq, a.n_tokens, a.q_stride) ||
        !make_map(&p.k, a.dtype, a.k, a.d, a.nkv, a.n_tokens, a.k_stride) ||
        !make_map(&p.v, a.dtype, a.v, a.d, a.nkv, a.n_tokens, a.v_stride))
        return cudaErrorInvalidValue;
    // one block per SM, fewer where there are fewer items: row blocks (at most
    // n_tokens / 128 and one more per sequence, or what max_len allows) times
    // half the heads, rounded up for an odd group
    const long long top = a.max_len < a.n_tokens ? a.max_len : a.n_tokens;
    long long blocks = a.n_tokens / kTile + a.n_seqs;
    const long long most = a.n_seqs * ((top + kTile - 1) / kTile);
    if (most < blocks) blocks = most;
    long long grid = blocks * ((a.nq / a.nkv + 1) / 2) * a.nkv;
    if (grid < 1) grid = 1;
    if (grid > num_sms) grid = num_sms;
    if (a.dtype == MK_BF16)
        return a.d == 64 ? launch<Bf16, 64>(p, device, (int)grid, stream)
                         : launch<Bf16, 128>(p, device, (int)grid, stream);
    return a.d == 64 ? launch<Fp16, 64>(p, device, (int)grid, stream)
                     : launch<Fp16, 128>(p, device, (int)grid, stream);
}

}  // namespace mk
