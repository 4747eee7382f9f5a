// mk_sample.cu -- sample a token per row of logits: temperature, top-k, top-p
// and min-p from given uniform numbers.
//
// One block per row, several passes over the row.  Logits are compared as
// ordered 32-bit keys; the cut of top-k (by count) and of top-p (by mass) is
// found by histograms of 2048 bins over a shrinking key range (32 -> 21 -> 10
// -> 0 bits left), so no sort is needed.  Weights are 64-bit integers in
// units of 2^-43 of the largest, which makes every sum exact and independent
// of its order.
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

__global__ void __launch_bounds__(kSampThreads) sample_kernel(SampleArgs a) {
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
    wt.inv_t = 1.0 / (double)t;
    wt.top = key_logit(top_key);
    const float mp = a.min_p ? a.min_p[row] : 0.f;
    wt.min_w = mp > 0.f ? fmin((double)mp, 1.0) : 0.0;
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

}  // namespace

cudaError_t sample_launch(const SampleArgs &a, int, int, cudaStream_t stream) {
    sample_kernel<<<a.rows, kSampThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace mk
