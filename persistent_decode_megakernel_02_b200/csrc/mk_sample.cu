// mk_sample.cu -- sample a token per row of logits: temperature, top-k, top-p
// and min-p from given uniform numbers.
//
// Logits are compared as ordered 32-bit keys, and weights are 64-bit integers
// in units of 2^-43 of the largest, which makes every sum exact and
// independent of its order (and of how a row is spread over blocks).
//
// A row goes to a cluster of 1 to 8 blocks, which hold it in shared memory
// from its one read to the end and exchange maxima, histograms and sums
// through each other's shared memory.  No sort:
//  - temperature and min-p alone: one exchange of sums, then the block, vector
//    step, warp, lane and element that hold uniform * total;
//  - top-k up to 384: the k-th largest of the threads' maxima is a lower bound
//    of the k-th largest logit that leaves few logits above it (about k /
//    (1 - k / 8192) of a row); those are gathered in block 0, which ranks them
//    pairwise and applies top-p and min-p to them alone;
//  - top-p alone: a histogram of masses over the distance from the largest
//    logit (128 bins per unit of l / T) gives the bin that holds the cut; its
//    logits are gathered and ranked, and the cut goes back to all blocks;
//  - what these leave over (larger k, many equal logits, very flat rows): the
//    exact cut by histograms over a shrinking key range (32 -> 21 -> 10 -> 0
//    bits left).
//
// Rows beyond 8 blocks' shared memory take one block each that rereads them.
//
// What bounds it: one row, the latency of its exchanges between blocks (2.3 us
// of load, then about 1 us an exchange): 9.3 us at 128256 logits with every
// filter, 26.6 with top-p alone; many rows, the 64-bit weights (12 cycles an SM
// for 32 of them) and the histogram's atomics of the rows that need them all:
// 64 mixed ones 42 us, 256 with top-k 101 us (1.3 TB/s), with top-p 300.
#include <atomic>
#include <utility>

#include <cooperative_groups.h>

#include "mk_ops.cuh"

namespace mk {
namespace {

constexpr int kSampThreads = 1024, kSampWarps = kSampThreads / 32, kBins = 2048;
typedef unsigned long long u64;

// Order-preserving key of a logit; 0 for -infinity and NaN (never chosen).
// -0 and +0 are equal.
__device__ __forceinline__ uint32_t logit_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    if ((u & 0x7fffffffu) > 0x7f800000u || u == 0xff800000u) return 0;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// Weights of a row.  2^(y / 32) for y = 32 (x - top) / (T ln 2) <= 0, as 2^n
// 2^(i / 32) 2^(r / 32): i from a table of 32, and |r| <= 1/2 by the Taylor
// polynomial of degree 4 (relative error (ln 2 / 64)^5 / 120 < 1.3e-12).
// Eleven 64-bit operations and no branch; the library's exp() made the passes
// that weigh a whole row twice as long.
constexpr double kMagic = 6755399441055744.0;     // 1.5 * 2^52: adding it rounds to an integer
constexpr double kTwo52 = 4503599627370496.0;     // the same, and a value below 2^52 becomes the low bits
constexpr u64 kTwo52Bits = 0x4330000000000000ull;
constexpr double kUnit = 8796093022208.0;         // 2^43
constexpr double kC = 0.021660849392498290;       // ln 2 / 32
struct Weight {
    double c32, top_d, min_v;    // y = c32 (x - top_d); min_v: min-p, in units
    // Logits below `reach` weigh nothing, below `floor` nothing in the final
    // choice; both are finite, so that -infinity is below them.
    float cap, reach, floor;
    const double *table;         // 2^(i / 32), shared memory

    __device__ __forceinline__ void init(const SampleArgs &a, int row, float top, float t, const double *tab) {
        c32 = 46.166241308446828384 / (double)t;  // 32 / ln 2
        cap = top == INFINITY ? 0.f : top;        // an infinite top and its equals weigh one
        top_d = (double)cap;
        float far = 31.2f;       // e^-31.2 < 2^-45
        const float mp = a.min_p ? a.min_p[row] : 0.f;
        min_v = 0.0;
        if (mp > 0.f) {
            min_v = fmin((double)mp, 1.0) * kUnit;
            far = fminf(far, fmaxf(-logf(mp), 0.f) * 1.0001f + 1e-4f);
        }
        const float lowest = -3.402823466e+38f;
        reach = fmaxf(top - 31.2f * t, lowest);
        floor = fmaxf(top - far * t, lowest);
        table = tab;
    }
    // 2^43 w, before rounding, of a logit that is not below `reach` (one that
    // is weighs less than half a unit)
    __device__ __forceinline__ double scaled(float x) const {
        const double y = ((double)fminf(fmaxf(x, reach), cap) - top_d) * c32;
        const double shifted = y + kMagic;
        const int n = __double2loint(shifted);
        const double d = y - (shifted - kMagic);
        double e = fma(d, kC * kC * kC * kC / 24, kC * kC * kC / 6);
        e = fma(d, e, kC * kC / 2);
        e = fma(d, e, kC);
        e = fma(d, e, 1.0);
        const double w = table[n & 31] * e;
        return __hiloint2double(__double2hiint(w) + (((n >> 5) + 43) << 20), __double2loint(w));
    }
    // the weight in units, plus kTwo52Bits
    __device__ __forceinline__ u64 units_raw(double v) const {      // v <= 2^43
        return (u64)__double_as_longlong(v + kTwo52);
    }
    __device__ __forceinline__ u64 whole(float x) const {
        return x < reach ? 0ull : units_raw(scaled(x)) - kTwo52Bits;
    }
    __device__ __forceinline__ bool enough(float x) const { return scaled(x) >= min_v; }
    // the weight in the final choice
    __device__ __forceinline__ u64 final_whole(float x) const {
        const double v = scaled(x);
        return x < floor || v < min_v ? 0ull : units_raw(v) - kTwo52Bits;
    }
};
__device__ __forceinline__ void fill_table(double *table) {
    if (threadIdx.x < 32) table[threadIdx.x] = exp2((double)threadIdx.x / 32);
}
__device__ __forceinline__ u64 goal_of(float u, u64 total) {
    return min((u64)((double)(u > 0.f ? fminf(u, 1.f) : 0.f) * (double)total), total - 1);
}

template <class V>
__device__ __forceinline__ V block_sum(V v, V *tmp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (lane == 0) tmp[warp] = v;
    __syncthreads();
    V s = 0;
    for (int w = 0; w < kSampWarps; ++w) s += tmp[w];
    return s;
}

// Exclusive prefix sum of each thread's v over the block.
template <class V>
__device__ __forceinline__ V block_scan(V v, V *tmp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    V x = v;
    for (int o = 1; o < 32; o <<= 1) {
        const V y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) tmp[warp] = x;
    __syncthreads();
    V before = 0;
    for (int w = 0; w < warp; ++w) before += tmp[w];
    return before + x - v;
}

struct SampShared {
    u64 mass[kBins];
    uint32_t cnt[kBins];
    u64 tmp64[kSampWarps];
    uint32_t tmp32[kSampWarps];
    double table[32];
    uint32_t bin;
    u64 mass_before;
    uint32_t cnt_before;
};

__global__ void __launch_bounds__(kSampThreads) sample_long_kernel(SampleArgs a) {
    __shared__ SampShared sh;
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float *x = a.logits + (long long)row * a.stride;
    const int V = a.vocab;

    fill_table(sh.table);
    // largest logit, lowest index first
    u64 best = 0;
    for (int i = tid; i < V; i += kSampThreads) {
        const uint32_t k = logit_key(x[i]);
        const u64 c = k ? (u64)k << 32 | (uint32_t)~i : 0;
        best = c > best ? c : best;
    }
    for (int o = 16; o > 0; o >>= 1) {
        const u64 c = __shfl_xor_sync(0xffffffffu, best, o);
        best = c > best ? c : best;
    }
    if (lane == 0) sh.tmp64[warp] = best;
    __syncthreads();
    for (int w = 0; w < kSampWarps; ++w) best = sh.tmp64[w] > best ? sh.tmp64[w] : best;
    __syncthreads();
    const float t = a.temperature ? a.temperature[row] : 1.f;
    if (best == 0 || !(t > 0.f)) {
        if (tid == 0) a.token[row] = best == 0 ? -1 : (int)~(uint32_t)best;
        return;
    }
    const uint32_t top_key = (uint32_t)(best >> 32);
    Weight wt;
    wt.init(a, row, key_logit(top_key), t, sh.table);
    const bool inf_top = top_key == 0xff800000u;
    // an infinite top leaves only its equals
    uint32_t cut = inf_top ? top_key : 1u;    // keys below are out
    uint32_t ties = 0xffffffffu;              // of keys equal to cut, this many (lowest indices) stay

    const int k = a.top_k ? a.top_k[row] : 0;
    const float p = a.top_p ? a.top_p[row] : 1.f;
    for (int stage = 0; stage < 2; ++stage) {
        const bool by_mass = stage == 1;
        if (by_mass ? !(p < 1.f) : !(k > 0 && k < V)) continue;
        double target = 0.0;    // by mass: the mass to hold
        if (by_mass) {
            u64 m = 0;
            uint32_t eq = 0;
            for (int i = tid; i < V; i += kSampThreads) {
                const uint32_t key = logit_key(x[i]);
                if (key > cut) m += wt.whole(x[i]);
                eq += key == cut;
            }
            const uint32_t n_eq = block_sum(eq, sh.tmp32);
            const u64 total = block_sum(m, sh.tmp64) + (cut > 1u ? (u64)min(n_eq, ties) * wt.whole(key_logit(cut)) : 0);
            target = (double)p * (double)total;
        }
        uint32_t lo = cut, hi = top_key;
        u64 mass_above = 0;
        uint32_t cnt_above = 0;
        while (true) {
            int sh_bits = 0;
            while ((hi - lo) >> sh_bits >= kBins) ++sh_bits;
            for (int i = tid; i < kBins; i += kSampThreads) { sh.mass[i] = 0; sh.cnt[i] = 0; }
            if (tid == 0) sh.bin = 0xffffffffu;
            __syncthreads();
            for (int i = tid; i < V; i += kSampThreads) {
                const uint32_t key = logit_key(x[i]);
                if (key < lo || key > hi) continue;
                const uint32_t b = (hi - key) >> sh_bits;
                atomicAdd(&sh.cnt[b], 1u);
                if (by_mass) atomicAdd(&sh.mass[b], wt.whole(x[i]));
            }
            __syncthreads();
            // the first bin (from the top) at which the running total reaches the target
            const uint32_t c0 = sh.cnt[2 * tid], c1 = sh.cnt[2 * tid + 1];
            const u64 m0 = sh.mass[2 * tid], m1 = sh.mass[2 * tid + 1];
            const uint32_t cb = cnt_above + block_scan(c0 + c1, sh.tmp32);
            const u64 mb = mass_above + block_scan(m0 + m1, sh.tmp64);
            auto reached = [&](uint32_t c, u64 m) {
                return by_mass ? (double)m >= target && c > 0 : c >= (uint32_t)k;
            };
            const bool r0 = reached(cb, mb), r1 = reached(cb + c0, mb + m0), r2 = reached(cb + c0 + c1, mb + m0 + m1);
            if (!r0 && r2) {
                sh.bin = 2 * tid + (r1 ? 0 : 1);
                sh.cnt_before = r1 ? cb : cb + c0;
                sh.mass_before = r1 ? mb : mb + m0;
            }
            __syncthreads();
            const uint32_t bin = sh.bin;
            if (bin == 0xffffffffu) break;     // fewer than k, or ties cut short the mass: all stay
            cnt_above = sh.cnt_before;
            mass_above = sh.mass_before;
            const uint32_t new_hi = hi - (bin << sh_bits);
            const u64 span = ((u64)1 << sh_bits) - 1;
            const uint32_t new_lo = (u64)(new_hi - lo) > span ? new_hi - (uint32_t)span : lo;
            const uint32_t old_cut = cut;
            hi = new_hi;
            lo = new_lo;
            if (lo == hi) {
                uint32_t need;
                if (by_mass) {
                    const double w = (double)wt.whole(key_logit(lo));
                    const double n = w > 0 ? ceil((target - (double)mass_above) / w) : 1.0;
                    need = n < 1.0 ? 1u : n > 4e9 ? 0xffffffffu : (uint32_t)n;
                } else
                    need = (uint32_t)k - cnt_above;
                cut = lo;
                ties = lo == old_cut ? min(ties, need) : need;
                break;
            }
            __syncthreads();
        }
        __syncthreads();
    }

    // final choice: warps own consecutive chunks of the row
    const int chunk = ((V + kSampWarps - 1) / kSampWarps + 31) & ~31;
    const int b = min(warp * chunk, V), e = min(b + chunk, V);
    const u64 u_cut = cut > 1u ? wt.final_whole(key_logit(cut)) : 0;
    u64 strict = 0;
    uint32_t eq = 0;
    for (int i = b + lane; i < e; i += 32) {
        const uint32_t key = logit_key(x[i]);
        if (key > cut) strict += wt.final_whole(x[i]);
        eq += key == cut;
    }
    for (int o = 16; o > 0; o >>= 1) {
        strict += __shfl_xor_sync(0xffffffffu, strict, o);
        eq += __shfl_xor_sync(0xffffffffu, eq, o);
    }
    if (lane == 0) { sh.tmp64[warp] = strict; sh.tmp32[warp] = eq; }
    __syncthreads();
    u64 total = 0, before = 0;
    uint32_t eq_seen = 0, eq_before = 0;
    for (int w = 0; w < kSampWarps; ++w) {
        if (w == warp) { before = total; eq_before = eq_seen; }
        const uint32_t keep = min(ties - min(ties, eq_seen), sh.tmp32[w]);
        total += sh.tmp64[w] + (u64)keep * u_cut;
        eq_seen += sh.tmp32[w];
    }
    const u64 mine = strict + (u64)min(ties - min(ties, eq_before), eq) * u_cut;
    const u64 goal = goal_of(a.uniform[row], total);
    if (goal < before || goal >= before + mine) return;
    u64 run = before;
    uint32_t tie_rank = eq_before;
    for (int i0 = b; i0 < e; i0 += 32) {
        const int i = i0 + lane;
        u64 w = 0;
        const uint32_t key = i < e ? logit_key(x[i]) : 0;
        const unsigned eqm = __ballot_sync(0xffffffffu, key == cut);
        if (key > cut) w = wt.final_whole(x[i]);
        else if (key == cut && tie_rank + __popc(eqm & ((1u << lane) - 1)) < ties)
            w = u_cut;
        u64 s = w;
        for (int o = 1; o < 32; o <<= 1) {
            const u64 y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, run + s > goal);
        if (hit) {
            if (lane == __ffs(hit) - 1) a.token[row] = i;
            return;
        }
        run += __shfl_sync(0xffffffffu, s, 31);
        tie_rank += __popc(eqm);
    }
}

// ---- rows held in the shared memory of a cluster ---------------------------

namespace cg = cooperative_groups;

constexpr int kRegThreads = 512, kRegWarps = kRegThreads / 32, kMaxCluster = 8;
constexpr int kListMax = 512;                  // gathered logits, at most
// top-k by the threads' maxima, at most (one row of 128256, against the exact
// cut: k = 50 10.3 and 32.3 us, 200 14.8 and 32.5, 384 24.6 and 32.8; 64 rows of
// 32000: 10.8 and 32.8, 19.5 and 33.4, 39.5 and 33.8).  Chosen for few rows: with
// 64 the two ways cross between 200 and 384, above which this one costs up to a
// sixth more, as the pairwise ranking grows with k^2 in every row's first block.
constexpr int kMaxK = 384;
constexpr int kVecStep = 4 * kRegThreads;      // logits of one vector step of a block
constexpr int kMaxIt = 22;                     // vector steps of a slice: 176 KB of logits
constexpr int kStepsForTwo = 10;               // with which two blocks fit an SM

struct RegShared {
    union {
        struct {
            u64 mass[kBins];
            uint32_t cnt[kBins];
        };
        uint32_t part[3][kBins];      // masses in three parts of 15, 14 and 14 bits
        u64 sums[kBins];              // and put together
        struct {
            float maxima[kMaxCluster * kRegThreads];
            uint32_t bins[kBins];
        };
        struct {                      // block 0, once all have gathered: the above is read by then
            u64 sorted[kListMax];
            ulonglong2 kept[kListMax];
        };
    };
    u64 list[kListMax];               // gathered logits: key, then lowest index first
    u64 sub[kRegWarps], step[kMaxIt], groups[kBins / 32];
    double table[32];
    // written by every block of the cluster, read by all
    u64 x_best[kMaxCluster], x_sum[kMaxCluster], x_mass[kMaxCluster];
    uint32_t x_cnt[kMaxCluster];
    u64 found_mass;
    uint32_t found_bin, found_before, found_cnt;
    float warp_top[kMaxCluster * kRegWarps];
    float top, cut;
    int edge;
    int32_t last;
    uint32_t list_n;
    u64 tmp64[kRegWarps];
    uint32_t tmp32[kRegWarps];
};

static_assert(sizeof(RegShared) + kMaxIt * kVecStep * 4 <= 227 * 1024, "a slice fits a block's shared memory");
static_assert(2 * (sizeof(RegShared) + kStepsForTwo * kVecStep * 4 + 1024) <= 228 * 1024, "two blocks an SM");

template <class V>
__device__ __forceinline__ V block_max(V v, V *tmp) {
    for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kRegWarps; ++w) v = max(v, tmp[w]);
    return v;
}
template <class V>
__device__ __forceinline__ V reg_block_sum(V v, V *tmp) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
    __syncthreads();
    V s = 0;
#pragma unroll
    for (int w = 0; w < kRegWarps; ++w) s += tmp[w];
    return s;
}

// Sort n <= 512 values of shared memory, descending, into `out`: each is
// counted against all (several threads a value where n leaves them) and put
// in its place.  Values are distinct.  (A bitonic sort of 64-bit values took
// twice as long at 20 to 200 of them: its steps are short and dependent.)
template <class V>
__device__ __forceinline__ void sort_descending(const V *in, V *out, int n) {
    const int per = n <= 64 ? 8 : n <= 128 ? 4 : n <= 256 ? 2 : 1;
    const int i = threadIdx.x / per;
    if ((threadIdx.x & ~31) / per < n) {       // warps without a value skip the count
        const V v = in[min(i, n - 1)];
        int place = 0;
#pragma unroll 8
        for (int j = threadIdx.x & (per - 1); j < n; j += per) place += in[j] > v;
        for (int o = per >> 1; o > 0; o >>= 1) place += __shfl_xor_sync(0xffffffffu, place, o);
        if (i < n && (threadIdx.x & (per - 1)) == 0) out[place] = v;
    }
    __syncthreads();
}
// Exclusive prefix sum over the block, and the total.
__device__ __forceinline__ u64 reg_block_scan(u64 v, u64 *tmp, u64 &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 x = v;
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) tmp[warp] = x;
    __syncthreads();
    u64 before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kRegWarps; ++w) {
        if (w == warp) before = all;
        all += tmp[w];
    }
    total = all;
    return before + x - v;
}

// With more rows than fit the device at once, those with top-p alone, which
// take about twice as long, come first: the row of cluster c in that order.
// Every cluster looks it up for itself, so only up to kOrderRows rows, whose
// parameters are a few loads side by side; with more the last rows are little
// of the whole.  64 rows of 151936 with eight slow ones last: 68.7 us in the
// rows' own order, 57.4 in this one; 128: 140 and 122; no slow ones among 128
// (what the look-up costs): 82 and 85.  Up to 256 rows: 132 and 95 at 128.
constexpr int kOrderRows = 128;
__device__ __forceinline__ int row_in_order(const SampleArgs &a, int c) {
    const int lane = threadIdx.x & 31;
    float p[kOrderRows / 32];
    int k[kOrderRows / 32];
#pragma unroll
    for (int i = 0; i < kOrderRows / 32; ++i) {
        const int r = i * 32 + lane;
        p[i] = r < a.rows ? a.top_p[r] : 1.f;
        k[i] = r < a.rows && a.top_k ? a.top_k[r] : 0;
    }
    unsigned slow[kOrderRows / 32];
#pragma unroll
    for (int i = 0; i < kOrderRows / 32; ++i)
        slow[i] = __ballot_sync(0xffffffffu, p[i] < 1.f && !(k[i] > 0 && k[i] < a.vocab));
    int row0 = 0, nth = 0;      // the nth of `among`, rows from row0
    unsigned among = 1;
#pragma unroll
    for (int pass = 0; pass < 2; ++pass)
#pragma unroll
        for (int i = 0; i < kOrderRows / 32; ++i) {
            const int there = min(a.rows - i * 32, 32);
            if (there <= 0) break;
            const unsigned m = (pass == 0 ? slow[i] : ~slow[i]) & (there == 32 ? 0xffffffffu : (1u << there) - 1);
            const int n = __popc(m);
            if (c >= 0 && c < n) {
                row0 = i * 32;
                nth = c;
                among = m;
            }
            c -= n;
        }
    const bool me = (among >> lane & 1u) && __popc(among & ((1u << lane) - 1)) == nth;
    return row0 + __ffs(__ballot_sync(0xffffffffu, me)) - 1;
}

// A block's slice of the row is 16 warps' parts of IT vector steps (4 logits a
// lane), so index order is (warp, step, lane, element).  A thread only ever
// reads the logits it stored; NaN is stored as -infinity.
__global__ void __launch_bounds__(kRegThreads, 2) sample_kernel(SampleArgs a, int IT, bool in_order) {
    extern __shared__ float4 xs[];
    __shared__ __align__(16) RegShared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int CL = cl.num_blocks(), rank = cl.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = a.vocab;
    const int row = in_order ? row_in_order(a, blockIdx.x / CL) : blockIdx.x / CL;
    const float *x = a.logits + (long long)row * a.stride;
    RegShared *home = cl.map_shared_rank(&sh, 0);

    auto started = cl.barrier_arrive();     // every block has, before the first write to another's memory
    fill_table(sh.table);
    if (tid == 0) {
        sh.list_n = 0;
        sh.edge = -1;
    }
    for (int i = tid; i < kBins; i += kRegThreads) sh.bins[i] = 0;
    const float t = a.temperature ? a.temperature[row] : 1.f;
    const int k = a.top_k ? a.top_k[row] : 0;
    const float p = a.top_p ? a.top_p[row] : 1.f;

    // ---- the slice.  Vectors start at the 16-byte boundary at or before the
    // row (`skew` logits before it).
    const int skew = (int)(((uintptr_t)x >> 2) & 3);
    const int base = rank * IT * kVecStep + warp * IT * 128 + lane * 4 - skew;    // the thread's first logit
    float best = -INFINITY;
    int best_it = 0;
#pragma unroll 8
    for (int it = 0; it < IT; ++it) {
        const int i = base + it * 128;
        float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (i >= 0 && i + 4 <= V) f = __ldcs(reinterpret_cast<const float4 *>(x + i));
        else {
            if (i >= 0 && i < V) f.x = x[i];
            if (i + 1 >= 0 && i + 1 < V) f.y = x[i + 1];
            if (i + 2 >= 0 && i + 2 < V) f.z = x[i + 2];
            if (i + 3 >= 0 && i + 3 < V) f.w = x[i + 3];
        }
        f.x = fmaxf(f.x, -INFINITY);      // the other operand where one is NaN
        f.y = fmaxf(f.y, -INFINITY);
        f.z = fmaxf(f.z, -INFINITY);
        f.w = fmaxf(f.w, -INFINITY);
        xs[it * kRegThreads + tid] = f;
        const float m = fmaxf(fmaxf(f.x, f.y), fmaxf(f.z, f.w));
        if (m > best) {
            best = m;
            best_it = it;
        }
    }
    // f(logit, index) for every logit of the thread
    auto each = [&](auto f) {
#pragma unroll 2
        for (int it = 0; it < IT; ++it) {
            const float4 q = xs[it * kRegThreads + tid];
            const int i = base + it * 128;
            f(q.x, i);
            f(q.y, i + 1);
            f(q.z, i + 2);
            f(q.w, i + 3);
        }
    };
    auto gather = [&](float f, int i) {
        const uint32_t at = atomicAdd(&home->list_n, 1u);
        if (at < kListMax) home->list[at] = (u64)logit_key(f) << 32 | (uint32_t)~i;
    };
    auto logit_of = [](u64 id) { return key_logit((uint32_t)(id >> 32)); };

    cl.barrier_wait(std::move(started));
    Weight wt;
    const bool by_k = k > 0 && k < V, by_p = p < 1.f;
    float top;

    if (by_k && k <= kMaxK && t > 0.f) {
        // ---- top-k by the threads' maxima
        home->maxima[rank * kRegThreads + tid] = best;
        const float wm = warp_max(best);
        if (lane < CL) cl.map_shared_rank(&sh, lane)->warp_top[rank * kRegWarps + warp] = wm;
        cl.sync();
        top = -INFINITY;
        for (int i = lane; i < CL * kRegWarps; i += 32) top = fmaxf(top, sh.warp_top[i]);
        top = warp_max(top);
        if (top == -INFINITY) {
            if (rank == 0 && tid == 0) a.token[row] = -1;
            return;
        }
        wt.init(a, row, top, t, sh.table);
        const float scale = fminf(64.f / t, 1e30f);
        auto bin_of = [&](float f) { return f == top ? 0 : (int)fminf((top - f) * scale, (float)(kBins - 1)); };
        if (rank == 0) {
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r)
                if (r < CL) {
                    const float m = sh.maxima[r * kRegThreads + tid];
                    if (m > -INFINITY) atomicAdd(&sh.bins[bin_of(m)], 1u);
                }
            __syncthreads();
            const uint4 c = reinterpret_cast<const uint4 *>(sh.bins)[tid];
            uint32_t s = c.x + c.y + c.z + c.w, run = s;
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += y;
            }
            if (lane == 31) sh.tmp32[warp] = run;
            __syncthreads();
            run -= s;
#pragma unroll
            for (int w = 0; w < kRegWarps; ++w) run += w < warp ? sh.tmp32[w] : 0;
            if (run < (uint32_t)k && run + s >= (uint32_t)k) {
                int b = 0;
                uint32_t y = run + c.x;
                if (y < (uint32_t)k) { b = 1; y += c.y; }
                if (y < (uint32_t)k) { b = 2; y += c.z; }
                if (y < (uint32_t)k) b = 3;
                for (int r = 0; r < CL; ++r) cl.map_shared_rank(&sh, r)->edge = 4 * tid + b;
            }
        }
        cl.sync();
        // at least k logits lie in the bins up to it (not the last: all the rest)
        const int edge = sh.edge;
        if (edge >= 0 && edge < kBins - 1 && top < INFINITY) {
            const float beyond = (float)(edge + 1);
            auto in = [&](float f) { return (top - f) * scale < beyond; };      // bin_of(f) <= edge
#pragma unroll 4
            for (int it = 0; it < IT; ++it) {
                const float4 q = xs[it * kRegThreads + tid];
                const int i = base + it * 128;
                if (!in(fmaxf(fmaxf(q.x, q.y), fmaxf(q.z, q.w)))) continue;
                if (in(q.x)) gather(q.x, i);
                if (in(q.y)) gather(q.y, i + 1);
                if (in(q.z)) gather(q.z, i + 2);
                if (in(q.w)) gather(q.w, i + 3);
            }
            cl.sync();
            const uint32_t n = home->list_n;
            if (n <= kListMax) {
                if (rank != 0) return;
                sort_descending(sh.list, sh.sorted, (int)n);
                const u64 id = tid < n ? sh.sorted[tid] : 0;
                u64 total;
                u64 w = tid < n && tid < k ? wt.whole(logit_of(id)) : 0;
                const u64 before = reg_block_scan(w, sh.tmp64, total);
                if (by_p && tid > 0 && !((double)before < (double)p * (double)total)) w = 0;
                if (wt.min_v > 0.0 && w > 0 && !wt.enough(logit_of(id))) w = 0;
                // what lies ahead in index order: the list again, as (~index, weight)
                if (tid < n) sh.kept[tid] = make_ulonglong2((uint32_t)id, w);
                u64 run = 0;
                const u64 kept = reg_block_sum(w, sh.tmp64);      // synchronises
                if (w) {
#pragma unroll 4
                    for (uint32_t j = 0; j < n; ++j) {
                        const ulonglong2 o = sh.kept[j];
                        run += o.x > (uint32_t)id ? o.y : 0;
                    }
                    const u64 goal = goal_of(a.uniform[row], kept);
                    if (goal >= run && goal < run + w) a.token[row] = (int)~(uint32_t)id;
                }
                cl.sync();      // the others have read the count (or are gone)
                return;
            }
        }
    } else {
        // ---- the row's largest, lowest index first
        u64 id = 0;
        if (best > -INFINITY) {
            const float4 q = xs[best_it * kRegThreads + tid];
            const int c = q.x == best ? 0 : q.y == best ? 1 : q.z == best ? 2 : 3;
            id = (u64)logit_key(best) << 32 | (uint32_t)~(base + best_it * 128 + c);
        }
        id = block_max(id, sh.tmp64);
        if (tid < CL) cl.map_shared_rank(&sh, tid)->x_best[rank] = id;
        cl.sync();
        for (int r = 0; r < CL; ++r) id = max(id, sh.x_best[r]);
        if (id == 0 || !(t > 0.f)) {
            if (rank == 0 && tid == 0) a.token[row] = id == 0 ? -1 : (int)~(uint32_t)id;
            return;      // the same for every block; nobody reads another's memory any more
        }
        top = logit_of(id);
        wt.init(a, row, top, t, sh.table);
    }

    // Kept so far: logits above `cut`, and those equal to it up to index
    // `last`.  An infinite top leaves only its equals.
    float cut = top == INFINITY ? INFINITY : -3.402823466e+38f;      // (-infinity is out)
    int32_t last = 0x7fffffff;

    // The histogram bins of all blocks (filled, not yet synchronised): the
    // first bin at which reached(count, mass) turns true over the running totals,
    // with its count and what lies before it, in sh.found_*.  False if none.
    auto find_bin = [&](auto reached, bool masses, uint32_t cnt0, u64 mass0) {
        cl.sync();
        // every block adds up its share of the bins, consecutive ones per thread
        const int share = kBins / CL, lo = rank * share, per = max(share / kRegThreads, 1);
        if (tid == 0) sh.found_bin = 0xffffffffu;
        uint32_t c[4] = {0, 0, 0, 0};
        u64 m[4] = {0, 0, 0, 0};
        uint32_t csum = 0;
        u64 msum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int b = tid * per + i;
            if (i < per && b < share) {
#pragma unroll
                for (int r = 0; r < kMaxCluster; ++r)
                    if (r < CL) {
                        const RegShared *o = cl.map_shared_rank(&sh, r);
                        c[i] += o->cnt[lo + b];
                        if (masses) m[i] += o->mass[lo + b];
                    }
            }
            csum += c[i];
            msum += m[i];
        }
        uint32_t cs = csum;
        u64 ms = msum;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, cs, o);
            const u64 z = __shfl_up_sync(0xffffffffu, ms, o);
            if (lane >= o) { cs += y; ms += z; }
        }
        if (lane == 31) { sh.tmp32[warp] = cs; sh.tmp64[warp] = ms; }
        __syncthreads();
        uint32_t ctot = 0, cb = cs - csum;      // of the block, and before this thread
        u64 mtot = 0, mb = ms - msum;
#pragma unroll
        for (int w = 0; w < kRegWarps; ++w) {
            if (w < warp) { cb += sh.tmp32[w]; mb += sh.tmp64[w]; }
            ctot += sh.tmp32[w];
            mtot += sh.tmp64[w];
        }
        if (tid < CL) {
            RegShared *o = cl.map_shared_rank(&sh, tid);
            o->x_cnt[rank] = ctot;
            o->x_mass[rank] = mtot;
        }
        cl.sync();
        cb += cnt0;
        mb += mass0;
        for (int r = 0; r < rank; ++r) {
            cb += sh.x_cnt[r];
            mb += sh.x_mass[r];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i < per && tid * per + i < share && !reached(cb, mb) && reached(cb + c[i], mb + m[i])) {
                for (int r = 0; r < CL; ++r) {
                    RegShared *o = cl.map_shared_rank(&sh, r);
                    o->found_bin = lo + tid * per + i;
                    o->found_before = cb;
                    o->found_cnt = c[i];
                    o->found_mass = mb;
                }
            }
            cb += c[i];
            mb += m[i];
        }
        cl.sync();
        return sh.found_bin != 0xffffffffu;
    };
    auto clear_bins = [&] {
        for (int i = tid; i < kBins; i += kRegThreads) { sh.mass[i] = 0; sh.cnt[i] = 0; }
        __syncthreads();
    };

    bool done_p = !by_p;
    if (by_p && !by_k && top < INFINITY) {
        // ---- top-p alone: masses by distance from the top
        const float scale = fminf(128.f / t, 1e30f);
        auto bin_of = [&](float f) { return f == top ? 0 : (int)fminf((top - f) * scale, (float)(kBins - 1)); };
        for (int i = tid; i < 3 * kBins; i += kRegThreads) sh.part[0][i] = 0;
        __syncthreads();
        // a block's sum of 45056 parts of 15 bits fits 32 bits.  The last bin
        // (16 units and more below the top) may hold most of a row: summed in
        // registers
        u64 rest = 0;
        each([&](float f, int) {
            if (f < wt.reach) return;
            const int b = bin_of(f);
            const u64 w = wt.units_raw(wt.scaled(f)) - kTwo52Bits;
            if (b == kBins - 1) rest += w;
            else {
                atomicAdd(&sh.part[0][b], (uint32_t)w & 0x7fffu);
                atomicAdd(&sh.part[1][b], (uint32_t)(w >> 15) & 0x3fffu);
                atomicAdd(&sh.part[2][b], (uint32_t)(w >> 29));
            }
        });
        rest = reg_block_sum(rest, sh.tmp64);
        if (tid < CL) cl.map_shared_rank(&sh, tid)->x_sum[rank] = rest;
        // The parts together, four consecutive bins a thread, and the sums of
        // groups of 32 bins.  Every block finds the group over all blocks, then
        // the bin in it, by itself (reading all blocks' bins took 15300 cycles
        // of the 69000 of one row).
        {
            const uint4 p0 = reinterpret_cast<const uint4 *>(sh.part[0])[tid], p1 = reinterpret_cast<const uint4 *>(sh.part[1])[tid],
                        p2 = reinterpret_cast<const uint4 *>(sh.part[2])[tid];
            const u64 m0 = p0.x + ((u64)p1.x << 15) + ((u64)p2.x << 29), m1 = p0.y + ((u64)p1.y << 15) + ((u64)p2.y << 29),
                      m2 = p0.z + ((u64)p1.z << 15) + ((u64)p2.z << 29), m3 = p0.w + ((u64)p1.w << 15) + ((u64)p2.w << 29);
            __syncthreads();
            reinterpret_cast<ulonglong2 *>(sh.sums)[2 * tid] = make_ulonglong2(m0, m1);
            reinterpret_cast<ulonglong2 *>(sh.sums)[2 * tid + 1] = make_ulonglong2(m2, m3);
            u64 group = m0 + m1 + m2 + m3;
            for (int o = 1; o < 8; o <<= 1) group += __shfl_xor_sync(0xffffffffu, group, o);
            if ((tid & 7) == 0) sh.groups[tid >> 3] = group;
        }
        if (tid == 0) sh.found_bin = 0xffffffffu;
        cl.sync();
        // the sum over the blocks of entry tid / 8, in all eight threads of it
        auto over_blocks = [&](auto entry_of) {
            u64 v = 0;
            const int b = tid & 7;
            if (b < CL) v = entry_of(cl.map_shared_rank(&sh, b));
            for (int o = 1; o < 8; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            return v;
        };
        const u64 group = over_blocks([&](const RegShared *o) { return o->groups[tid >> 3]; });
        u64 all;
        const u64 group_at = reg_block_scan(tid & 7 ? 0 : group, sh.tmp64, all);      // exclusive: right in the first of eight
        for (int r = 0; r < CL; ++r) all += sh.x_sum[r];
        const double target = (double)p * (double)all;
        auto reached = [&](u64 mass) { return mass > 0 && (double)mass >= target; };    // the top is in bin 0
        if ((tid & 7) == 0 && !reached(group_at) && reached(group_at + group)) {
            sh.found_bin = tid >> 3;
            sh.found_mass = group_at;
        }
        __syncthreads();
        const uint32_t in_group = sh.found_bin;
        const u64 before_group = sh.found_mass;      // read before the scan: it is written again after it
        if (in_group != 0xffffffffu) {
            const u64 mass = over_blocks([&](const RegShared *o) { return tid < 256 ? o->sums[in_group * 32 + (tid >> 3)] : 0; });
            u64 sum;
            const u64 at = before_group + reg_block_scan(tid & 7 ? 0 : mass, sh.tmp64, sum);      // synchronises
            if (tid < 256 && (tid & 7) == 0 && !reached(at) && reached(at + mass)) {
                sh.found_bin = in_group * 32 + (tid >> 3);
                sh.found_mass = at;
            }
            __syncthreads();
        }
        if (sh.found_bin != 0xffffffffu) {
            const int bin = (int)sh.found_bin;
            each([&](float f, int i) {
                if (bin_of(f) == bin) gather(f, i);
            });
            cl.sync();
            if (rank == 0) {
                const uint32_t n = sh.list_n;
                float c = -INFINITY;
                int l = -1;
                if (n <= kListMax) {
                    sort_descending(sh.list, sh.sorted, (int)n);
                    const u64 id = tid < n ? sh.sorted[tid] : 0;
                    u64 total;
                    const u64 before = reg_block_scan(tid < n ? wt.whole(logit_of(id)) : 0, sh.tmp64, total);
                    const bool keep = tid < n && ((tid == 0 && bin == 0) || (double)(sh.found_mass + before) < target);
                    // the kept ones come first: the last of them is the cut
                    const uint32_t kept = reg_block_sum(keep ? 1u : 0u, sh.tmp32);
                    if (keep && tid == kept - 1) {
                        sh.cut = logit_of(id);
                        sh.last = (int)~(uint32_t)id;
                    }
                    __syncthreads();
                    c = sh.cut;
                    l = sh.last;
                    __syncthreads();
                }
                if (tid < CL) {
                    RegShared *o = cl.map_shared_rank(&sh, tid);
                    o->cut = c;
                    o->last = l;
                }
            }
            cl.sync();
            if (sh.last >= 0) {
                cut = sh.cut;
                last = sh.last;
                done_p = true;
            }
        }
        cl.sync();      // the sums and the cut are read
    }

    // The index at which the running sum of weight(logit, index), in index
    // order, first exceeds goal(total).  One thread of the cluster calls
    // done(index).  Logits below `least` weigh nothing.
    auto pick = [&](float least, auto weight, auto goal, auto done) {
        u64 s = 0;
        if (least > wt.reach) {
            // a part of the row: of 32 logits a thread those that are in it, two at a
            // time (64 mixed rows 42.8 -> 41.7 us against all four of a vector with one)
#pragma unroll 1
            for (int it0 = 0; it0 < IT; it0 += 8) {
                uint32_t in = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (it0 + j < IT) {
                        const float4 q = xs[(it0 + j) * kRegThreads + tid];
                        in |= ((q.x >= least ? 1u : 0u) | (q.y >= least ? 2u : 0u) | (q.z >= least ? 4u : 0u) | (q.w >= least ? 8u : 0u))
                              << 4 * j;
                    }
                while (in) {
                    int i[2];
                    float f[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int b = __ffs(in) - 1, it = it0 + (b >> 2);
                        f[j] = -INFINITY;
                        i[j] = 0;
                        if (b >= 0) {
                            f[j] = reinterpret_cast<const float *>(xs)[(it * kRegThreads + tid) * 4 + (b & 3)];
                            i[j] = base + it * 128 + (b & 3);
                        }
                        in &= in - 1;
                    }
                    s += weight(f[0], i[0]) + weight(f[1], i[1]);
                }
            }
        } else
#pragma unroll 2
            for (int it = 0; it < IT; ++it) {
                const float4 q = xs[it * kRegThreads + tid];
                const int i = base + it * 128;
                s += weight(q.x, i) + weight(q.y, i + 1) + weight(q.z, i + 2) + weight(q.w, i + 3);
            }
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        __syncthreads();
        if (lane == 0) sh.sub[warp] = s;
        __syncthreads();
        u64 mine = 0;
#pragma unroll
        for (int w = 0; w < kRegWarps; ++w) mine += sh.sub[w];
        if (tid < CL) cl.map_shared_rank(&sh, tid)->x_sum[rank] = mine;
        cl.sync();
        u64 total = 0, run = 0;
        for (int r = 0; r < CL; ++r) {
            if (r == rank) run = total;
            total += sh.x_sum[r];
        }
        const u64 g = goal(total);
        if (g < run || g >= run + mine) return;       // not in this block
        // the warp's part that holds it; its steps are weighed by a warp each
        // (by the part's own warp, one step after another, it took 8000 cycles)
        int part = 0;
#pragma unroll
        for (int w = 0; w < kRegWarps - 1; ++w)
            if (part == w && g >= run + sh.sub[w]) {
                run += sh.sub[w];
                part = w + 1;
            }
        const int first = rank * IT * kVecStep + part * IT * 128 + lane * 4 - skew;
        u64 own[4];
        auto step_sum = [&](int it) {       // up to and with this lane
            const float4 q = xs[it * kRegThreads + part * 32 + lane];
            const int i = first + it * 128;
            own[0] = weight(q.x, i);
            own[1] = weight(q.y, i + 1);
            own[2] = weight(q.z, i + 2);
            own[3] = weight(q.w, i + 3);
            u64 at = own[0] + own[1] + own[2] + own[3];
            for (int o = 1; o < 32; o <<= 1) {
                const u64 y = __shfl_up_sync(0xffffffffu, at, o);
                if (lane >= o) at += y;
            }
            return at;
        };
        for (int it = warp; it < IT; it += kRegWarps) {
            const u64 at = step_sum(it);
            if (lane == 31) sh.step[it] = at;
        }
        __syncthreads();
        if (warp != 0) return;
        int it = 0;
        while (it < IT - 1 && g >= run + sh.step[it]) run += sh.step[it++];
        u64 at = run + step_sum(it);
        for (int c = 3; c >= 0; --c) {
            at -= own[c];
            if (g >= at && g < at + own[c]) done(first + it * 128 + c);
        }
    };

    // ---- the exact cuts, by count and by mass, where nothing above found them
    for (int stage = 0; stage < 2; ++stage) {
        const bool by_mass = stage == 1;
        if (by_mass ? done_p : !by_k) continue;
        double target = 0.0;
        if (by_mass) {
            u64 m = 0;
            each([&](float f, int i) {
                if (f > cut || (f == cut && i <= last)) m += wt.whole(f);
            });
            m = reg_block_sum(m, sh.tmp64);
            cl.sync();
            if (tid < CL) cl.map_shared_rank(&sh, tid)->x_sum[rank] = m;
            cl.sync();
            u64 total = 0;
            for (int r = 0; r < CL; ++r) total += sh.x_sum[r];
            target = (double)p * (double)total;
            cl.sync();
        }
        uint32_t lo = max(logit_key(cut), 1u), hi = logit_key(top), cnt_above = 0;
        u64 mass_above = 0;
        while (true) {
            int bits = 0;
            while ((hi - lo) >> bits >= kBins) ++bits;
            clear_bins();
            each([&](float f, int i) {
                const uint32_t ky = logit_key(f);
                if (ky < lo || ky > hi || (f == cut && i > last)) return;
                const uint32_t b = (hi - ky) >> bits;
                atomicAdd(&sh.cnt[b], 1u);
                if (by_mass) atomicAdd(&sh.mass[b], wt.whole(f));
            });
            if (!find_bin(
                    [&](uint32_t c, u64 m) { return by_mass ? c > 0 && (double)m >= target : c >= (uint32_t)k; },
                    by_mass, cnt_above, mass_above))
                break;      // fewer than k: all stay
            cnt_above = sh.found_before;
            mass_above = sh.found_mass;
            hi -= sh.found_bin << bits;
            const u64 span = ((u64)1 << bits) - 1;
            if ((u64)(hi - lo) > span) lo = hi - (uint32_t)span;
            if (lo != hi) continue;
            uint32_t need = (uint32_t)k - cnt_above;      // of the equal ones
            if (by_mass) {
                const double w = (double)wt.whole(key_logit(lo));
                const double n = w > 0 ? ceil((target - (double)mass_above) / w) : 1.0;
                need = n < 1.0 ? 1u : n > 4e9 ? 0xffffffffu : (uint32_t)n;
            }
            const int32_t old = key_logit(lo) == cut ? last : 0x7fffffff;
            cut = key_logit(lo);
            last = old;
            if (need < sh.found_cnt) {     // up to the need-th in index order
                cl.sync();
                pick(cut, [&](float f, int i) { return f == cut && i <= old ? 1ull : 0ull; },
                     [&](u64) { return (u64)need - 1; },
                     [&](int i) {
                         for (int r = 0; r < CL; ++r) cl.map_shared_rank(&sh, r)->last = i;
                     });
                cl.sync();
                last = sh.last;
            }
            break;
        }
    }

    const float u = a.uniform[row];
    const float least = fmaxf(cut, wt.floor);
    pick(least, [&](float f, int i) { return f < cut || (f == cut && i > last) ? 0ull : wt.final_whole(f); },
         [&](u64 total) { return goal_of(u, total); }, [&](int i) { a.token[row] = i; });
    cl.sync();    // nobody leaves while its memory may still be written
}

}  // namespace

cudaError_t sample_launch(const SampleArgs &a, int device, int num_sms, cudaStream_t stream) {
    // Up to eight blocks a row, as many as get a vector step each; fewer where
    // that brings all rows onto the device at once and two blocks still fit an
    // SM (64 rows of 32000, 8 and 4 blocks a row: top-k 20.1 and 10.8 us, top-p
    // 44 and 28; one row: 8.2 and 8.7, 17 and 20).  (Up to 3 logits lie ahead of
    // a row that starts inside a 16-byte word.)
    const int need = a.vocab + 3;
    auto steps_of = [&](int blocks) { return (need + blocks * kVecStep - 1) / (blocks * kVecStep); };
    int cluster = 1;
    while (cluster < kMaxCluster && steps_of(cluster) > 1) cluster *= 2;
    while (cluster > 1 && (long long)a.rows * cluster > 2 * num_sms && steps_of(cluster / 2) <= kStepsForTwo) cluster /= 2;
    const int steps = steps_of(cluster);
    if (steps > kMaxIt) return launch_kernel(sample_long_kernel, a.rows, kSampThreads, 0, stream, a);
    static std::atomic<bool> ready[kOpsMaxDevices];
    if (!ready[device].load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kMaxIt * kVecStep * 4);
        if (e != cudaSuccess) return e;
        ready[device].store(true, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.rows * cluster);
    cfg.blockDim = dim3(kRegThreads);
    cfg.dynamicSmemBytes = (size_t)steps * kVecStep * 4;
    cfg.stream = stream;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cluster;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    const bool in_order = a.top_p && (long long)a.rows * cluster > 2 * num_sms && a.rows <= kOrderRows;
    return cudaLaunchKernelEx(&cfg, sample_kernel, a, steps, in_order);
}

}  // namespace mk
