// mk_sample.cu -- sample a token per row of logits: temperature, top-k, top-p
// and min-p from given uniform numbers.
//
// Logits are compared as ordered 32-bit keys, and weights are 64-bit integers
// in units of 2^-43 of the largest, which makes every sum exact and
// independent of its order (and of how a row is spread over blocks).
//
// A row goes to a cluster of 1 to 8 blocks, which hold it in
// shared memory from its one read to the end; the blocks exchange maxima, histograms and
// sums through each other's shared memory.  A row without top-k and top-p is
// one exchange of sums.  Top-k and top-p first find, by a histogram over the
// distance from the largest logit (64 bins per unit of l / T), the bin that
// holds the cut; when at most 512 candidates lie above its lower edge they are
// gathered in one block, which ranks them pairwise and finishes alone.
// Otherwise (flat rows, very large k) the cut is found exactly by histograms
// over a shrinking key range (32 -> 21 -> 10 -> 0 bits left).  No sort.
//
// Rows beyond 8 blocks' shared memory take one block each that rereads them.
#include <atomic>

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

struct Weight {
    double inv_t;
    float top;      // the row's largest logit
    double min_w;   // min-p: weights below it are dropped from the final choice
    // w = exp((x - top) / T); x is neither NaN nor -infinity
    __device__ __forceinline__ double real(float x) const {
        return x == top ? 1.0 : exp(((double)x - (double)top) * inv_t);
    }
    __device__ __forceinline__ u64 whole(double w) const { return (u64)(w * 8796093022208.0); }   // 2^43
    __device__ __forceinline__ void init(const SampleArgs &a, int row, uint32_t top_key, float t) {
        inv_t = 1.0 / (double)t;
        top = key_logit(top_key);
        const float mp = a.min_p ? a.min_p[row] : 0.f;
        min_w = mp > 0.f ? fmin((double)mp, 1.0) : 0.0;
    }
};

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
    uint32_t bin;
    u64 mass_before, mass_bin;
    uint32_t cnt_before, cnt_bin;
};

__global__ void __launch_bounds__(kSampThreads) sample_long_kernel(SampleArgs a) {
    __shared__ SampShared sh;
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float *x = a.logits + (long long)row * a.stride;
    const int V = a.vocab;

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
    wt.init(a, row, top_key, t);
    const bool inf_top = isinf(wt.top);
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
                if (key > cut) m += wt.whole(wt.real(x[i]));
                eq += key == cut;
            }
            const uint32_t n_eq = block_sum(eq, sh.tmp32);
            const u64 total = block_sum(m, sh.tmp64) + (u64)min(n_eq, ties) * wt.whole(wt.real(key_logit(cut)));
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
                if (by_mass) atomicAdd(&sh.mass[b], wt.whole(wt.real(x[i])));
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
                sh.cnt_bin = r1 ? c0 : c1;
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
                    const double w = (double)wt.whole(wt.real(key_logit(lo)));
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
    const double w_cut = cut > 1u ? wt.real(key_logit(cut)) : 0.0;
    const u64 u_cut = w_cut >= wt.min_w ? wt.whole(w_cut) : 0;
    u64 strict = 0;
    uint32_t eq = 0;
    for (int i = b + lane; i < e; i += 32) {
        const uint32_t key = logit_key(x[i]);
        if (key > cut) {
            const double w = wt.real(x[i]);
            if (w >= wt.min_w) strict += wt.whole(w);
        }
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
    const float u = a.uniform[row];
    u64 goal = (u64)((double)(u > 0.f ? fminf(u, 1.f) : 0.f) * (double)total);
    goal = min(goal, total - 1);
    if (goal < before || goal >= before + mine) return;
    u64 run = before;
    uint32_t tie_rank = eq_before;
    for (int i0 = b; i0 < e; i0 += 32) {
        const int i = i0 + lane;
        u64 w = 0;
        const uint32_t key = i < e ? logit_key(x[i]) : 0;
        const unsigned eqm = __ballot_sync(0xffffffffu, key == cut);
        if (key > cut) {
            const double f = wt.real(x[i]);
            if (f >= wt.min_w) w = wt.whole(f);
        } else if (key == cut && tie_rank + __popc(eqm & ((1u << lane) - 1)) < ties)
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

constexpr int kRegThreads = 512, kRegWarps = kRegThreads / 32, kMaxCluster = 8, kListMax = 512;
constexpr int kVecStep = 4 * kRegThreads;      // logits of one vector step of a block
constexpr int kMaxIt = 22;                     // vector steps of a slice: 176 KB of logits

struct RegShared {
    u64 mass[kBins];
    uint32_t cnt[kBins];
    u64 list_w[kListMax], list_keep[kListMax];
    uint32_t list_key[kListMax];
    int32_t list_idx[kListMax];
    u64 sub[kMaxIt * kRegWarps];          // sums per (vector step, warp)
    // written by every block of the cluster, read by all
    u64 x_best[kMaxCluster], x_sum[kMaxCluster], x_mass[kMaxCluster];
    uint32_t x_cnt[kMaxCluster];
    u64 found_mass;
    uint32_t found_bin, found_before, found_cnt;
    int32_t tie_last;
    uint32_t list_n;
    u64 tmp64[kRegWarps];
    uint32_t tmp32[kRegWarps];
    u64 goal;
    int hit;
};

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

// A block's slice of the row is IT vector steps of 4 logits a thread, kept as
// keys: vector (it, thread) holds logits 4 (it * 512 + thread).. of the slice,
// so index order is (it, warp, lane, element).  A thread only ever reads the
// keys it wrote.
__global__ void __launch_bounds__(kRegThreads) sample_kernel(SampleArgs a, int IT) {
    extern __shared__ uint4 keys[];
    __shared__ RegShared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int CL = cl.num_blocks(), rank = cl.block_rank();
    const int row = blockIdx.x / CL, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float *x = a.logits + (long long)row * a.stride;
    const int V = a.vocab;

    // ---- the slice, as keys; 0 beyond the row.  Vectors start at the 16-byte
    // boundary at or before the row (`skew` logits before it).
    const int skew = (int)(((uintptr_t)x >> 2) & 3);
    const int base = rank * IT * kVecStep - skew;       // index of the slice's first logit
    u64 best = 0;      // the largest key, lowest index first
#pragma unroll 4
    for (int it = 0; it < IT; ++it) {
        const int i = base + it * kVecStep + 4 * tid;
        float4 f = make_float4(NAN, NAN, NAN, NAN);
        if (i >= 0 && i + 4 <= V) f = __ldcs(reinterpret_cast<const float4 *>(x + i));
        else {
            if (i >= 0 && i < V) f.x = x[i];
            if (i + 1 >= 0 && i + 1 < V) f.y = x[i + 1];
            if (i + 2 >= 0 && i + 2 < V) f.z = x[i + 2];
            if (i + 3 >= 0 && i + 3 < V) f.w = x[i + 3];
        }
        uint4 q;
        q.x = logit_key(f.x);
        q.y = logit_key(f.y);
        q.z = logit_key(f.z);
        q.w = logit_key(f.w);
        keys[it * kRegThreads + tid] = q;
        const uint32_t m = max(max(q.x, q.y), max(q.z, q.w));
        if (m > (uint32_t)(best >> 32)) {
            const int c = q.x == m ? 0 : q.y == m ? 1 : q.z == m ? 2 : 3;
            best = (u64)m << 32 | (uint32_t)~(i + c);
        }
    }
    // f(key, index) for every logit of the thread
    auto each = [&](auto f) {
#pragma unroll 1
        for (int it = 0; it < IT; ++it) {
            const uint4 q = keys[it * kRegThreads + tid];
            const int i = base + it * kVecStep + 4 * tid;
            f(q.x, i);
            f(q.y, i + 1);
            f(q.z, i + 2);
            f(q.w, i + 3);
        }
    };
    const float t = a.temperature ? a.temperature[row] : 1.f;
    const int k = a.top_k ? a.top_k[row] : 0;
    const float p = a.top_p ? a.top_p[row] : 1.f;

    // ---- the row's largest
    for (int o = 16; o > 0; o >>= 1) {
        const u64 c = __shfl_xor_sync(0xffffffffu, best, o);
        best = c > best ? c : best;
    }
    if (lane == 0) sh.tmp64[warp] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kRegWarps; ++w) best = sh.tmp64[w] > best ? sh.tmp64[w] : best;
    if (tid < CL) cl.map_shared_rank(&sh, tid)->x_best[rank] = best;
    if (tid == 0) sh.list_n = 0;
    cl.sync();
    for (int r = 0; r < CL; ++r) best = sh.x_best[r] > best ? sh.x_best[r] : best;
    if (best == 0 || !(t > 0.f)) {
        if (rank == 0 && tid == 0) a.token[row] = best == 0 ? -1 : (int)~(uint32_t)best;
        return;      // the same for every block; nobody reads another's memory any more
    }
    const uint32_t top_key = (uint32_t)(best >> 32);
    Weight wt;
    wt.init(a, row, top_key, t);
    uint32_t cut = isinf(wt.top) ? top_key : 1u;   // keys below are out
    uint32_t ties = 0xffffffffu;                   // of keys equal to cut, this many (lowest indices) stay
    const bool by_k = k > 0 && k < V, by_p = p < 1.f;

    // The histogram bins of all blocks (filled, not yet synchronised): the
    // first bin at which the running (count, mass) reaches the target, with
    // what lies before it.  False if none does.  *all_mass: everything's mass.
    auto find_bin = [&](auto reached, bool masses, uint32_t cnt0, u64 mass0, u64 *all_mass) {
        cl.sync();
        // every block adds up its share of the bins
        const int share = kBins / CL, lo = rank * share;
        if (tid == 0) sh.found_bin = 0xffffffffu;
        uint32_t c[4] = {0, 0, 0, 0};      // consecutive bins per thread: share <= 4 * 512
        u64 m[4] = {0, 0, 0, 0};
        const int per = (share + kRegThreads - 1) / kRegThreads;
        uint32_t csum = 0;
        u64 msum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int b = tid * per + i;
            if (i < per && b < share) {
                for (int r = 0; r < CL; ++r) {
                    const RegShared *o = cl.map_shared_rank(&sh, r);
                    c[i] += o->cnt[lo + b];
                    if (masses) m[i] += o->mass[lo + b];
                }
            }
            csum += c[i];
            msum += m[i];
        }
        // exclusive scan over the block
        uint32_t cs = csum;
        u64 ms = msum;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, cs, o);
            const u64 z = __shfl_up_sync(0xffffffffu, ms, o);
            if (lane >= o) { cs += y; ms += z; }
        }
        if (lane == 31) { sh.tmp32[warp] = cs; sh.tmp64[warp] = ms; }
        __syncthreads();
        uint32_t ctot = 0, cb = cs - csum;
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
        u64 total = mass0;
        for (int r = 0; r < CL; ++r) {
            if (r < rank) { cb += sh.x_cnt[r]; mb += sh.x_mass[r]; }
            total += sh.x_mass[r];
        }
        if (all_mass) *all_mass = total;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i < per && tid * per + i < share && !reached(cb, mb, total) && reached(cb + c[i], mb + m[i], total)) {
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

    if ((by_k || by_p) && !isinf(wt.top)) {
        // ---- candidates by distance from the top: 64 bins per unit of l / T
        const float scale = fminf(64.f / t, 1e30f);
        auto bin_of = [&](uint32_t ky) { return (int)fminf((wt.top - key_logit(ky)) * scale, (float)(kBins - 1)); };
        clear_bins();
        each([&](uint32_t ky, int) {
            if (!ky) return;
            const int b = bin_of(ky);
            atomicAdd(&sh.cnt[b], 1u);
            if (!by_k) atomicAdd(&sh.mass[b], wt.whole(wt.real(key_logit(ky))));
        });
        u64 all = 0;
        const bool found = find_bin(
            [&](uint32_t c, u64 m, u64 total) {
                return by_k ? c >= (uint32_t)k : c > 0 && (double)m >= (double)p * (double)total;
            },
            !by_k, 0, 0, &all);
        const uint32_t n = sh.found_before + sh.found_cnt;
        if (found && n <= kListMax && sh.found_bin < kBins - 1) {
            // ---- gather them in block 0
            RegShared *home = cl.map_shared_rank(&sh, 0);
            const int edge = (int)sh.found_bin;
            each([&](uint32_t ky, int i) {
                if (!ky || bin_of(ky) > edge) return;
                const uint32_t at = atomicAdd(&home->list_n, 1u);
                home->list_key[at] = ky;
                home->list_idx[at] = i;
            });
            cl.sync();
            if (rank != 0) return;
            if (tid < n) {
                sh.list_w[tid] = wt.whole(wt.real(key_logit(sh.list_key[tid])));
            }
            __syncthreads();
            // rank and mass before, pairwise: one candidate per thread
            uint32_t place = 0;
            u64 before = 0, w = 0;
            uint32_t ky = 0;
            int32_t idx = 0;
            if (tid < n) {
                ky = sh.list_key[tid];
                idx = sh.list_idx[tid];
                w = sh.list_w[tid];
                for (uint32_t j = 0; j < n; ++j) {
                    const uint32_t kj = sh.list_key[j];
                    if (kj > ky || (kj == ky && sh.list_idx[j] < idx)) {
                        ++place;
                        before += sh.list_w[j];
                    }
                }
            }
            bool keep = tid < n && (!by_k || place < (uint32_t)k);
            if (by_p) {
                const u64 total = by_k ? reg_block_sum(keep ? w : 0ull, sh.tmp64) : all;
                keep = keep && (place == 0 || (double)before < (double)p * (double)total);
            }
            keep = keep && (wt.min_w == 0.0 || wt.real(key_logit(ky)) >= wt.min_w);
            if (!keep) w = 0;
            if (tid < n) sh.list_keep[tid] = w;
            const u64 total = reg_block_sum(w, sh.tmp64);     // synchronises
            const float u = a.uniform[row];
            const u64 goal = min((u64)((double)(u > 0.f ? fminf(u, 1.f) : 0.f) * (double)total), total - 1);
            if (w > 0) {
                u64 run = 0;
                for (uint32_t j = 0; j < n; ++j)
                    if (sh.list_idx[j] < idx) run += sh.list_keep[j];
                if (run <= goal && goal < run + w) a.token[row] = idx;
            }
            return;
        }
        // ---- the exact cuts, by count and by mass
        for (int stage = 0; stage < 2; ++stage) {
            const bool by_mass = stage == 1;
            if (by_mass ? !by_p : !by_k) continue;
            double target = 0.0;
            if (by_mass) {
                u64 m = 0;
                uint32_t eq = 0;
                each([&](uint32_t ky, int) {
                    if (ky > cut) m += wt.whole(wt.real(key_logit(ky)));
                    eq += ky == cut;
                });
                const u64 bm = reg_block_sum(m, sh.tmp64);
                const uint32_t be = reg_block_sum(eq, sh.tmp32);
                cl.sync();
                if (tid < CL) {
                    RegShared *o = cl.map_shared_rank(&sh, tid);
                    o->x_sum[rank] = bm;
                    o->x_cnt[rank] = be;
                }
                cl.sync();
                u64 total = 0;
                uint32_t n_eq = 0;
                for (int r = 0; r < CL; ++r) { total += sh.x_sum[r]; n_eq += sh.x_cnt[r]; }
                total += cut > 1u ? (u64)min(n_eq, ties) * wt.whole(wt.real(key_logit(cut))) : 0;
                target = (double)p * (double)total;
                cl.sync();
            }
            uint32_t lo = cut, hi = top_key, cnt_above = 0;
            u64 mass_above = 0;
            while (true) {
                int bits = 0;
                while ((hi - lo) >> bits >= kBins) ++bits;
                clear_bins();
                each([&](uint32_t ky, int) {
                    if (ky < lo || ky > hi) return;
                    const uint32_t b = (hi - ky) >> bits;
                    atomicAdd(&sh.cnt[b], 1u);
                    if (by_mass) atomicAdd(&sh.mass[b], wt.whole(wt.real(key_logit(ky))));
                });
                if (!find_bin([&](uint32_t c, u64 m, u64) { return by_mass ? c > 0 && (double)m >= target : c >= (uint32_t)k; },
                              by_mass, cnt_above, mass_above, nullptr))
                    break;      // fewer than k, or ties cut short the mass: all stay
                cnt_above = sh.found_before;
                mass_above = sh.found_mass;
                hi -= sh.found_bin << bits;
                const u64 span = ((u64)1 << bits) - 1;
                if ((u64)(hi - lo) > span) lo = hi - (uint32_t)span;
                if (lo == hi) {
                    uint32_t need = (uint32_t)k - cnt_above;
                    if (by_mass) {
                        const double w = (double)wt.whole(wt.real(key_logit(lo)));
                        const double n = w > 0 ? ceil((target - (double)mass_above) / w) : 1.0;
                        need = n < 1.0 ? 1u : n > 4e9 ? 0xffffffffu : (uint32_t)n;
                    }
                    ties = lo == cut ? min(ties, need) : need;
                    cut = lo;
                    break;
                }
            }
        }
    }

    // The index at which the running sum of weight(e, index), in index order,
    // first exceeds the goal; goal_of(total) gives it.  One thread of the
    // cluster calls done(index).
    auto pick = [&](auto weight, auto goal_of, auto done) {
        __syncthreads();
#pragma unroll 1
        for (int it = 0; it < IT; ++it) {
            const uint4 q = keys[it * kRegThreads + tid];
            const int i = base + it * kVecStep + 4 * tid;
            u64 s = weight(q.x, i) + weight(q.y, i + 1) + weight(q.z, i + 2) + weight(q.w, i + 3);
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == 0) sh.sub[it * kRegWarps + warp] = s;
        }
        __syncthreads();
        // warp 0: sums over (it, warp), N consecutive ones a lane
        const int N = (IT * kRegWarps + 31) / 32;
        if (warp == 0) {
            u64 s = 0;
            for (int i = 0; i < N; ++i) s += lane * N + i < IT * kRegWarps ? sh.sub[lane * N + i] : 0;
            u64 run = s;
            for (int o = 1; o < 32; o <<= 1) {
                const u64 y = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += y;
            }
            const u64 mine = __shfl_sync(0xffffffffu, run, 31);
            if (lane < CL) cl.map_shared_rank(&sh, lane)->x_sum[rank] = mine;
            sh.tmp64[0] = mine;
        }
        cl.sync();
        u64 total = 0, before = 0;
        for (int r = 0; r < CL; ++r) {
            if (r == rank) before = total;
            total += sh.x_sum[r];
        }
        const u64 goal = goal_of(total);
        const bool here = goal >= before && goal < before + sh.x_sum[rank];
        if (here) {       // the same answer for the whole block
            if (warp == 0) {
                u64 s = 0;
                for (int i = 0; i < N; ++i) s += lane * N + i < IT * kRegWarps ? sh.sub[lane * N + i] : 0;
                u64 run = s;
                for (int o = 1; o < 32; o <<= 1) {
                    const u64 y = __shfl_up_sync(0xffffffffu, run, o);
                    if (lane >= o) run += y;
                }
                run += before - s;
                for (int i = 0; i < N; ++i) {
                    const u64 w = lane * N + i < IT * kRegWarps ? sh.sub[lane * N + i] : 0;
                    if (goal >= run && goal < run + w) {
                        sh.hit = lane * N + i;
                        sh.goal = goal - run;
                    }
                    run += w;
                }
            }
            __syncthreads();
            if (sh.hit % kRegWarps == warp) {
                const int it = sh.hit / kRegWarps, i = base + it * kVecStep + 4 * tid;
                const uint4 q = keys[it * kRegThreads + tid];
                const u64 w[4] = {weight(q.x, i), weight(q.y, i + 1), weight(q.z, i + 2), weight(q.w, i + 3)};
                u64 run = w[0] + w[1] + w[2] + w[3];
                const u64 mine = run;
                for (int o = 1; o < 32; o <<= 1) {
                    const u64 y = __shfl_up_sync(0xffffffffu, run, o);
                    if (lane >= o) run += y;
                }
                run -= mine;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (sh.goal >= run && sh.goal < run + w[c]) done(i + c);
                    run += w[c];
                }
            }
        }
    };

    int32_t last = 0x7fffffff;    // ties up to this index stay
    if (ties != 0xffffffffu) {
        if (tid == 0) sh.tie_last = 0x7fffffff;
        cl.sync();
        pick([&](uint32_t ky, int) { return ky == cut ? 1ull : 0ull; }, [&](u64) { return (u64)ties - 1; },
             [&](int i) {
                 for (int r = 0; r < CL; ++r) cl.map_shared_rank(&sh, r)->tie_last = i;
             });
        cl.sync();
        last = sh.tie_last;
    }
    const float u = a.uniform[row];
    pick(
        [&](uint32_t ky, int i) {
            if (ky < cut || ky == 0 || (ky == cut && i > last)) return 0ull;
            const double w = wt.real(key_logit(ky));
            return w >= wt.min_w ? wt.whole(w) : 0ull;
        },
        [&](u64 total) {
            return min((u64)((double)(u > 0.f ? fminf(u, 1.f) : 0.f) * (double)total), total - 1);
        },
        [&](int i) { a.token[row] = i; });
    cl.sync();    // nobody leaves while its memory may still be written
}

}  // namespace

cudaError_t sample_launch(const SampleArgs &a, int device, int, cudaStream_t stream) {
    // Eight blocks a row from 8 vector steps each on; shorter rows take fewer.
    // (up to 3 logits ahead of a row that starts inside a 16-byte word)
    const int need = a.vocab + 3;
    int cluster = 1;
    while (cluster < kMaxCluster && need > cluster * kVecStep) cluster *= 2;
    const int steps = (need + cluster * kVecStep - 1) / (cluster * kVecStep);
    if (steps > kMaxIt) {
        sample_long_kernel<<<a.rows, kSampThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
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
    return cudaLaunchKernelEx(&cfg, sample_kernel, a, steps);
}

}  // namespace mk
