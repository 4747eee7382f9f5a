// mk_paged_attn.cu -- attention of one new token per sequence over a paged
// cache, split over the caches' length and joined in the same launch.
//
// Every key and value is read once for the G query heads of its KV head; 4 G
// flops per 4 bytes, so the kernel is bound by memory as long as enough bytes
// are in flight.  The work of all (sequence, KV head) items is laid end to
// end in steps of 8 KB of cache and cut into equal ranges, one per block:
// ragged batches and single long sequences balance alike.  The warps of a
// block take the steps of an item in turn, each with its own softmax state;
// states are merged through shared memory, and where an item spans several
// blocks the partial states go to the workspace and the block that finishes
// last merges them in block order (results do not depend on who is last).
//
// The products run on the tensor cores straight from registers, with keys
// and head dims as the long sides and heads as the short one:
//   S^T[16 keys][8 heads] = K Q^T,   O^T[16 dims][8 heads] += V^T P^T
// (mma m16n8k16).  A lane loads 16-byte pieces of K rows (its row, a quarter
// of each 32 dims) and V rows (its four keys, an eighth of each 64 dims): the
// order of the dims within the contraction is free, so the pieces are the
// fragments, and V needs one byte permute per register.  Nothing is staged in
// shared memory.  tcgen05 would need the rows staged and 128-row tiles with
// at most 8 useful columns; at 16 flops a byte the kernel is far below the
// tensor rate either way.
//
// The softmax weights enter the value product as a 16-bit value and the
// 16-bit remainder, in two products.  In bf16 the two hold a weight to 2^-16 of
// itself.  In fp16 they hold it to 2^-22, but nothing below 2^-25: so the
// weights are scaled to at most 2^15 there, and what is lost of one is at most
// 2^-40 of a warp's largest (with the largest at 1 to 2^8, as in bf16, 8192 keys
// at 2^-20 of the largest were off by 3 % and vanished below 2^-25).
//
// What bounds it: 203000 positions in 32 sequences of 8 x 128 take 128 us,
// 6.5 TB/s, 99 % of the copy rate.  At 34 MB (16 sequences of up to 2048, one
// of 16385: 14.3 and 12.9 us, 5.2 by the copy rate) the chain of dependent
// latencies around the stream does: lengths, page table, first rows, and the
// merge through the workspace; one sequence of 551 is that chain alone, 7.1 us.
#include "mk_ops.cuh"

namespace mk {
namespace {

constexpr int kMaxBlocksPerSm = 2;
// An item costs a block about this many steps whatever its length (one
// 128-position item a block: 4.7 us in all, 17 items of 2 steps one after
// another 30 us).  4 / 8 / 16 / 24: 64 ragged sequences of up to 1000 33, 25, 24,
// 25 us, 16 of up to 2048 15.2, 15.0, 13.6, 14.6.
constexpr int kItemCost = 16;

__device__ __forceinline__ uint4 ld_stream(const uint16_t *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
template <class T>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if constexpr (T::kBf16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8x8 transpose of 16-bit elements across the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t word(const uint4 &v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// A warp's reference maximum is raised when a score exceeds it by more than
// kHead powers of two, and a weight is 2^(score - reference + kScale).  (In fp16
// every rise raises it, or two powers of headroom and a scale of 2^13: 147 and
// 147 us for 32 ragged sequences of up to 16384, 8 x 128, 12.5 and 12.5 for 16 of
// up to 2048, 8 x 64.)
template <class T>
struct PagedWeight {
    static constexpr float kHead = T::kBf16 ? 8.f : 0.f, kScale = T::kBf16 ? 0.f : 15.f;
};

template <int D>
struct PagedShape {
    static constexpr int kGran = D == 64 ? 2 : 1;    // 16-key groups per step
    static constexpr int kStep = 16 * kGran;         // keys per step: 8 KB of K and V
    // least part of an item (one sequence of 551 and one of 4096 positions, 8 KV
    // heads: 64 dims 4 steps 6.7 and 9.9 us, 8 7.6 and 9.2, 16 8.4 and 10.3; 128
    // dims 8 steps 9.1 and 13.2, 16 9.7 and 11.2, 24 12.9 and 12.8)
    static constexpr int kMinSteps = D == 64 ? 4 : 16;
    static constexpr int kWarps = D == 64 ? 8 : 6;
    static constexpr int kThreads = kWarps * 32;
};

// Workspace: one counter per block (zero between calls), then two partial
// states per block: [8 heads][D] sums, [8][2] maxima and sums of weights.
__host__ __device__ constexpr size_t slot_floats(int d) { return (size_t)MK_MAX_GROUP * d + 2 * MK_MAX_GROUP; }
__host__ __device__ constexpr size_t counter_bytes(int blocks) { return ((size_t)blocks * 4 + 255) & ~(size_t)255; }

struct PagedParams {
    PagedArgs a;
    int max_blocks;      // counters in the workspace
};

template <class T, int D>
__global__ void __launch_bounds__(PagedShape<D>::kThreads, 2) paged_attn_kernel(const __grid_constant__ PagedParams p) {
    using S = PagedShape<D>;
    using W = PagedWeight<T>;
    constexpr int NW = S::kWarps, NT = S::kThreads, KG = S::kGran, JK = D / 32, JV = D / 64;
    __shared__ float so[NW][MK_MAX_GROUP][D];
    __shared__ float sm[NW][MK_MAX_GROUP], sl[NW][MK_MAX_GROUP];
    __shared__ int s_last;
    const PagedArgs &a = p.a;
    const int nkv = a.kv.n_kv_heads, G = a.n_q_heads / nkv, ps = a.kv.page_size, ns = a.kv.n_seqs;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int P = gridDim.x, blk = blockIdx.x;
    const float c = a.scale * 1.4426950408889634f;
    uint32_t *counters = (uint32_t *)a.workspace;
    float *slots = (float *)((char *)a.workspace + counter_bytes(p.max_blocks));

    auto clamped = [&](int n) { return min(max(n, 0), a.max_len); };
    auto steps_of = [&](int n) { return (n + S::kStep - 1) / S::kStep; };

    // ---- this block's part of the work: all items end to end, each with
    // kItemCost steps ahead of its own, cut into equal ranges.  (A second rule
    // for few items, equal parts of one item a block, was slower by 0.4 us at
    // one sequence of 551 and of 16385 positions and at 16 of up to 2048.)
    const int n0 = lane < ns ? a.lens[lane] : 0;
    auto len_of = [&](int s0) { return s0 == 0 ? clamped(n0) : s0 + lane < ns ? clamped(a.lens[s0 + lane]) : 0; };
    int total = 0, items = 0;
    for (int s0 = 0; s0 < ns; s0 += 32) {
        const int n = len_of(s0);
        total += steps_of(n);
        items += n > 0;
    }
    for (int o = 16; o > 0; o >>= 1) {
        total += __shfl_xor_sync(0xffffffffu, total, o);
        items += __shfl_xor_sync(0xffffffffu, items, o);
    }
    const int all_items = items * nkv;
    total *= nkv;
    total += all_items * kItemCost;
    const int per = max((total - 1) / P + 1, S::kMinSteps);
    const int lo = min(blk * per, total);   // blk * per < total + P * kMinSteps
    const int hi = min(total, lo + per);
    auto cost_of = [&](int n) { return n <= 0 ? 0 : steps_of(n) + kItemCost; };

    // empty sequences get zeros; lengths outside the bounds are reported
    auto empties = [&] {
        for (int s = blk; s < ns; s += P) {
            const int n = a.lens[s];
            if (n < 0 || n > a.max_len) bad_value(a.status);
            if (clamped(n) == 0)
                for (int i = tid; i < a.n_q_heads * D / 8; i += NT)
                    *reinterpret_cast<uint4 *>((uint16_t *)a.out + s * a.out_stride + i * 8) = make_uint4(0, 0, 0, 0);
        }
    };
    // ---- the sequence holding step lo
    int seq = 0, len = 0;
    int seq0 = 0;   // first step of the sequence
    bool found = false;
    for (int s0 = 0; s0 < ns && !found; s0 += 32) {
        const int n = len_of(s0);
        const int mine = cost_of(n) * nkv;
        int sum = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, seq0 + sum > lo);
        if (hit) {
            const int src = __ffs(hit) - 1;
            seq = s0 + src;
            len = __shfl_sync(0xffffffffu, n, src);
            seq0 += __shfl_sync(0xffffffffu, sum - mine, src);
            found = true;
        } else
            seq0 += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (!found) {
        empties();
        return;
    }

    int cur = lo;
    while (true) {
        const int steps = steps_of(len), cost = cost_of(len);
        const int h = (cur - seq0) / cost;
        // steps [b, e) of the item; its parts are blocks first..
        const int item0 = seq0 + h * cost + kItemCost;   // its first step
        const int b = max(cur - item0, 0), e = min(hi, item0 + steps) - item0;
        const int first = item0 / per, parts = (item0 + steps - 1) / per - first + 1;
        cur = item0 + steps;
        if (e > b) {

        // queries of this KV head: lane (g, t) holds head g's elements
        // [(4 j + t) 8, +8)
        uint4 q[JK];
        {
            const uint16_t *src = (const uint16_t *)a.q + seq * a.q_stride + (long long)(h * G + g) * D + t * 8;
#pragma unroll
            for (int j = 0; j < JK; ++j)
                q[j] = g < G ? *reinterpret_cast<const uint4 *>(src + j * 32) : make_uint4(0, 0, 0, 0);
        }
        float acc[JV * 4][4];
#pragma unroll
        for (int i = 0; i < JV * 4; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[i][k] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};   // heads 2t, 2t + 1

        const int32_t *table = a.kv.page_table + (long long)seq * a.kv.pages_per_seq;
        // cache row of this lane's key of a step; -1: not there
        auto row_of = [&](int i) {
            const int pos = i * S::kStep + lane % S::kStep;
            if (i >= e || pos >= len) return -1;
            const int page = table[pos / ps];
            if (page < 0 || page >= a.kv.num_pages) {
                bad_value(a.status);
                return -1;
            }
            return (page * nkv + h) * ps + pos % ps;
        };
        uint4 kr[KG][2][JK], vr[KG][4][JV];
        auto load_k = [&](int row) {
#pragma unroll
            for (int r = 0; r < KG; ++r)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int rr = __shfl_sync(0xffffffffu, row, r * 16 + x * 8 + g);
                    const uint16_t *src = (const uint16_t *)a.kv.k + (long long)rr * D + t * 8;
#pragma unroll
                    for (int j = 0; j < JK; ++j)
                        kr[r][x][j] = rr >= 0 ? ld_stream(src + j * 32) : make_uint4(0, 0, 0, 0);
                }
        };
        auto load_v = [&](int row) {
#pragma unroll
            for (int r = 0; r < KG; ++r)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int rr = __shfl_sync(0xffffffffu, row, r * 16 + (x >> 1) * 8 + 2 * t + (x & 1));
                    const uint16_t *src = (const uint16_t *)a.kv.v + (long long)rr * D + g * 8;
#pragma unroll
                    for (int j = 0; j < JV; ++j)
                        vr[r][x][j] = rr >= 0 ? ld_stream(src + j * 64) : make_uint4(0, 0, 0, 0);
                }
        };

        int i = b + warp;
        int row = row_of(i), next = row_of(i + NW);
        if (i < e) {
            load_k(row);
            load_v(row);
        }
        for (; i < e; i += NW) {
            // scores, keys g and g + 8 of each group, heads 2t and 2t + 1
            float s[KG][4];
#pragma unroll
            for (int r = 0; r < KG; ++r) {
                s[r][0] = s[r][1] = s[r][2] = s[r][3] = 0.f;
#pragma unroll
                for (int j = 0; j < JK; ++j) {
                    mma16816<T>(s[r], kr[r][0][j].x, kr[r][1][j].x, kr[r][0][j].y, kr[r][1][j].y, q[j].x, q[j].y);
                    mma16816<T>(s[r], kr[r][0][j].z, kr[r][1][j].z, kr[r][0][j].w, kr[r][1][j].w, q[j].z, q[j].w);
                }
            }
            const int after = row_of(i + 2 * NW);
            load_k(next);
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int r = 0; r < KG; ++r)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const bool there = __shfl_sync(0xffffffffu, row, r * 16 + x * 8 + g) >= 0;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        s[r][2 * x + k] = there ? s[r][2 * x + k] * c : -INFINITY;
                        top[k] = fmaxf(top[k], s[r][2 * x + k]);
                    }
                }
#pragma unroll
            for (int k = 0; k < 2; ++k)
                for (int o = 4; o < 32; o <<= 1) top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], o));
            const bool up = top[0] > m[0] + W::kHead || top[1] > m[1] + W::kHead;
            if (__any_sync(0xffffffffu, up)) {
                float f[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float n = fmaxf(m[k], top[k]);
                    f[k] = n == m[k] ? 1.f : ex2(m[k] - n);
                    m[k] = n;
                    l[k] *= f[k];
                }
#pragma unroll
                for (int y = 0; y < JV * 4; ++y)
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[y][k] *= f[k & 1];
            }
            const float m0 = m[0] == -INFINITY ? 0.f : m[0], m1 = m[1] == -INFINITY ? 0.f : m[1];
#pragma unroll
            for (int r = 0; r < KG; ++r) {
                uint32_t hi2[2], lo2[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float w0 = ex2(s[r][2 * x] - m0 + W::kScale), w1 = ex2(s[r][2 * x + 1] - m1 + W::kScale);
                    l[0] += w0;
                    l[1] += w1;
                    const uint32_t wh = T::pack(w0, w1);
                    const float2 back = T::unpack(wh);
                    const uint32_t wl = T::pack(w0 - back.x, w1 - back.y);
                    hi2[x] = transpose8(wh);
                    lo2[x] = transpose8(wl);
                }
#pragma unroll
                for (int j = 0; j < JV; ++j)
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint32_t v0 = word(vr[r][0][j], y), v1 = word(vr[r][1][j], y), v2 = word(vr[r][2][j], y),
                                       v3 = word(vr[r][3][j], y);
                        const uint32_t a0 = __byte_perm(v0, v1, 0x5410), a1 = __byte_perm(v0, v1, 0x7632),
                                       a2 = __byte_perm(v2, v3, 0x5410), a3 = __byte_perm(v2, v3, 0x7632);
                        mma16816<T>(acc[j * 4 + y], a0, a1, a2, a3, hi2[0], hi2[1]);
                        mma16816<T>(acc[j * 4 + y], a0, a1, a2, a3, lo2[0], lo2[1]);
                    }
            }
            load_v(next);
            row = next;
            next = after;
        }

#pragma unroll
        for (int k = 0; k < 2; ++k)
            for (int o = 4; o < 32; o <<= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], o);

        // ---- an infinite value times a remainder that is zero or negative made
        // a NaN of what is infinite: look at the values again and put it right.
        // (A second run of the loop with such values taken out of the remainders'
        // product cost every call 7 to 15 %.)
        bool nan = false;
#pragma unroll
        for (int y = 0; y < JV * 4; ++y)
#pragma unroll
            for (int k = 0; k < 4; ++k) nan |= acc[y][k] != acc[y][k];
        if (__any_sync(0xffffffffu, nan)) {
            uint32_t seen[3] = {0, 0, 0};     // NaN, +inf, -inf in this lane's columns, a bit each
#pragma unroll 1
            for (i = b + warp; i < e; i += NW) {
                load_v(row_of(i));
#pragma unroll
                for (int r = 0; r < KG; ++r)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
#pragma unroll
                        for (int j = 0; j < JV; ++j)
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const float2 v = T::unpack(word(vr[r][x][j], y));
                                const uint32_t at = 1u << (j * 8 + 2 * y);
                                seen[0] |= (v.x != v.x ? at : 0) | (v.y != v.y ? 2 * at : 0);
                                seen[1] |= (v.x == INFINITY ? at : 0) | (v.y == INFINITY ? 2 * at : 0);
                                seen[2] |= (v.x == -INFINITY ? at : 0) | (v.y == -INFINITY ? 2 * at : 0);
                            }
            }
#pragma unroll
            for (int kind = 0; kind < 3; ++kind)
                for (int o = 1; o < 4; o <<= 1) seen[kind] |= __shfl_xor_sync(0xffffffffu, seen[kind], o);
#pragma unroll
            for (int y = 0; y < JV * 4; ++y)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t at = 1u << (2 * y + (k >> 1));
                    // (a NaN among the scores, or no score above -infinity: NaN all over)
                    if (l[k & 1] == l[k & 1] && m[k & 1] > -INFINITY && !(seen[0] & at) && ((seen[1] ^ seen[2]) & at))
                        acc[y][k] = seen[1] & at ? INFINITY : -INFINITY;
                }
        }

        // ---- merge the warps' states
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (g == 0) {
                sm[warp][2 * t + k] = m[k];
                sl[warp][2 * t + k] = l[k];
            }
#pragma unroll
            for (int j = 0; j < JV; ++j)
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    *reinterpret_cast<float2 *>(&so[warp][2 * t + k][(j * 8 + g) * 8 + 2 * y]) =
                        make_float2(acc[j * 4 + y][k], acc[j * 4 + y][2 + k]);
        }
        __syncthreads();
        const bool whole = b == 0 && e == steps;
        // an item's first block keeps its part in slot 1 (its last item), later ones in slot 0
        float *slot = slots + (size_t)(2 * blk + (b == 0)) * slot_floats(D);
        for (int idx = tid; idx < G * D / 2; idx += NT) {
            const int hd = idx / (D / 2), x = idx % (D / 2) * 2;
            float M = -INFINITY, L = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) M = fmaxf(M, sm[w][hd]);
            const float M0 = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float f = ex2(sm[w][hd] - M0);   // 0 for a warp that saw nothing
                L += f * sl[w][hd];
                o0 += f * so[w][hd][x];
                o1 += f * so[w][hd][x + 1];
            }
            if (whole) {
                const float inv = L == 0.f ? 0.f : 1.f / L;
                *reinterpret_cast<uint32_t *>((uint16_t *)a.out + seq * a.out_stride + (long long)(h * G + hd) * D +
                                              x) = T::pack(o0 * inv, o1 * inv);
            } else {
                *reinterpret_cast<float2 *>(slot + hd * D + x) = make_float2(o0, o1);
                if (x == 0) *reinterpret_cast<float2 *>(slot + MK_MAX_GROUP * D + hd * 2) = make_float2(M, L);
            }
        }
        if (!whole) {
            // ---- the block that finishes an item last joins its parts
            __syncthreads();   // the block's part is written; the counter's release covers it
            if (tid == 0) s_last = atom_add_acqrel_gpu(&counters[first], 1u) == (uint32_t)parts - 1;
            __syncthreads();
            if (s_last) {
                if (tid == 0) counters[first] = 0;   // ready for the next call
                auto part = [&](int i) { return slots + (size_t)(2 * (first + i) + (i == 0)) * slot_floats(D); };
                // a thread takes four columns of every groups-th part, with a
                // running maximum; the groups' results meet in shared memory
                const int cols = G * D / 4, groups = max(1, NT / cols);
                float4 *red = reinterpret_cast<float4 *>(&so[0][0][0]);             // [groups][cols]
                float2 *ml = reinterpret_cast<float2 *>(&so[0][0][0]) + 2 * NT;      // the same, M and L
                for (int idx = tid; idx < cols * groups; idx += NT) {
                    const int col = idx % cols, grp = idx / cols, hd = col / (D / 4);
                    float M = -INFINITY, L = 0.f;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int i = grp; i < parts; i += groups) {
                        const float2 x = __ldcg(reinterpret_cast<const float2 *>(part(i) + MK_MAX_GROUP * D + hd * 2));
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(part(i)) + col);
                        const float n = fmaxf(M, x.x), N = n == -INFINITY ? 0.f : n;
                        const float f = ex2(M - N), w = ex2(x.x - N);
                        M = n;
                        L = L * f + w * x.y;
                        o.x = o.x * f + w * v.x;
                        o.y = o.y * f + w * v.y;
                        o.z = o.z * f + w * v.z;
                        o.w = o.w * f + w * v.w;
                    }
                    red[idx] = o;
                    if (groups > 1) ml[idx] = make_float2(M, L);
                    else {
                        const float inv = L == 0.f ? 0.f : 1.f / L;
                        red[idx] = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
                    }
                }
                __syncthreads();
                for (int col = tid; col < cols; col += NT) {
                    float4 o = red[col];
                    if (groups > 1) {
                        float M = -INFINITY, L = 0.f;
                        for (int grp = 0; grp < groups; ++grp) M = fmaxf(M, ml[grp * cols + col].x);
                        const float M0 = M == -INFINITY ? 0.f : M;
                        o = make_float4(0.f, 0.f, 0.f, 0.f);
                        for (int grp = 0; grp < groups; ++grp) {
                            const float4 v = red[grp * cols + col];
                            const float2 x = ml[grp * cols + col];
                            const float w = ex2(x.x - M0);
                            L += w * x.y;
                            o.x += w * v.x; o.y += w * v.y; o.z += w * v.z; o.w += w * v.w;
                        }
                        const float inv = L == 0.f ? 0.f : 1.f / L;
                        o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
                    }
                    uint2 w;
                    w.x = T::pack(o.x, o.y);
                    w.y = T::pack(o.z, o.w);
                    *reinterpret_cast<uint2 *>((uint16_t *)a.out + seq * a.out_stride + (long long)h * G * D +
                                               col * 4) = w;
                }
            }
        }
        __syncthreads();   // the shared states are free again

        }
        // ---- next item of the range
        if (cur >= hi) break;
        while (cur >= seq0 + cost_of(len) * nkv) {
            seq0 += cost_of(len) * nkv;
            len = clamped(a.lens[++seq]);
        }
    }
    empties();
}

}  // namespace

static int max_blocks(int num_sms) { return kMaxBlocksPerSm * num_sms; }

static int grid_of(const mk_paged_kv &kv, int max_len, int num_sms) {
    const int least = kv.head_dim == 64 ? PagedShape<64>::kStep * PagedShape<64>::kMinSteps
                                        : PagedShape<128>::kStep * PagedShape<128>::kMinSteps;
    const long long want = (long long)kv.n_seqs * kv.n_kv_heads * ((max_len + least - 1) / least);
    return (int)(want < 1 ? 1 : want > max_blocks(num_sms) ? max_blocks(num_sms) : want);
}

size_t paged_workspace(const mk_paged_kv &kv, int max_len, int num_sms) {
    return counter_bytes(max_blocks(num_sms)) +
           (size_t)grid_of(kv, max_len, num_sms) * 2 * slot_floats(kv.head_dim) * sizeof(float);
}

template <class T, int D>
static cudaError_t paged_go(const PagedParams &p, int grid, cudaStream_t stream) {
    return launch_kernel(paged_attn_kernel<T, D>, grid, PagedShape<D>::kThreads, 0, stream, p);
}

cudaError_t paged_launch(const PagedArgs &a, int num_sms, cudaStream_t stream) {
    PagedParams p{a, max_blocks(num_sms)};
    const int grid = grid_of(a.kv, a.max_len, num_sms);
    if (a.kv.dtype == MK_BF16)
        return a.kv.head_dim == 64 ? paged_go<Bf16, 64>(p, grid, stream) : paged_go<Bf16, 128>(p, grid, stream);
    return a.kv.head_dim == 64 ? paged_go<Fp16, 64>(p, grid, stream) : paged_go<Fp16, 128>(p, grid, stream);
}

}  // namespace mk
