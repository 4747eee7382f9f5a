// mk_kv_append.cu -- append rotated keys and values to a paged cache.
//
// For every new token: q' = R(pos) q, k' = R(pos) k with the half-split
// rotation of the decode step, k' and v into the cache row of the token's
// position.  Per token it reads (nq + 2 nkv) d elements and writes (nq +
// 2 nkv) d (and nkv d more with k_out), 3 flops each: bound by memory.
//
// A block takes TB consecutive tokens.  Its warps first look up the tokens'
// sequences, check their places, and fill a table of cos / sin in shared
// memory, one angle per (token, pair): pos * theta^(-2i/d) / (2 pi) in 64
// bits with the whole turns dropped, so that positions of any size keep
// their angle, then one 32-bit sincospi.  Then a thread takes a 16-byte pair of
// vectors (elements i.. and i + d/2..) of one head for all of the block's
// tokens, so that its loads are in flight together.
#include "mk_ops.cuh"

namespace mk {
namespace {

constexpr int kAppendThreads = 256;

struct AppendParams {
    AppendArgs a;
    double turn[64];   // theta^(-2i/d) / (2 pi)
};

struct Place {
    long long row;     // element offset of (page, head 0, row) in the cache
    int ok;
};

template <class T>
__device__ __forceinline__ void rotate(uint4 &x, uint4 &y, const float2 *cs) {
    uint32_t *px = &x.x, *py = &y.x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 a = T::unpack(px[j]), b = T::unpack(py[j]);
        const float2 c0 = cs[2 * j], c1 = cs[2 * j + 1];
        px[j] = T::pack(fmaf(a.x, c0.x, -b.x * c0.y), fmaf(a.y, c1.x, -b.y * c1.y));
        py[j] = T::pack(fmaf(b.x, c0.x, a.x * c0.y), fmaf(b.y, c1.x, a.y * c1.y));
    }
}

template <class T, int D, int TB>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int kHalf = D / 2, kVecs = kHalf / 8;   // 16-byte vectors in half a head
    __shared__ float2 cs[TB][kHalf];
    __shared__ Place place[TB];
    const AppendArgs &a = p.a;
    const long long t0 = (long long)blockIdx.x * TB;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nkv = a.kv.n_kv_heads, ps = a.kv.page_size;

    for (int i = warp; i < TB; i += kAppendThreads / 32) {
        Place w{0, 0};
        int pos = 0;
        const long long t = t0 + i;
        if (t < a.n_tokens && t < a.cu[a.kv.n_seqs]) {
            const int s = warp_find_seq(a.cu, a.kv.n_seqs, (int)t);
            const long long at = (long long)a.start[s] + (t - a.cu[s]);
            bool ok = a.cu[s] >= 0 && t >= a.cu[s] && t < a.cu[s + 1] && at >= 0 &&
                      at < (long long)a.kv.pages_per_seq * ps;
            if (ok) {
                pos = (int)at;
                const int page = a.kv.page_table[(long long)s * a.kv.pages_per_seq + pos / ps];
                ok = page >= 0 && page < a.kv.num_pages;
                w.row = ((long long)page * nkv * ps + pos % ps) * D;
            }
            w.ok = ok;
            if (!ok && lane == 0) bad_value(a.status);
        }
        if (w.ok)
            for (int j = lane; j < kHalf; j += 32) {
                const double turns = (double)pos * p.turn[j];
                float sn, cn;
                sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cn);
                cs[i][j] = make_float2(cn, sn);
            }
        if (lane == 0) place[i] = w;
    }
    __syncthreads();

    // vector v of a head of every token; heads are q, then k, then v
    const int heads = a.n_q_heads + 2 * nkv;
    for (int r = threadIdx.x; r < heads * kVecs; r += kAppendThreads) {
        const int head = r / kVecs, v = r % kVecs;
        const bool is_q = head < a.n_q_heads, is_k = !is_q && head < a.n_q_heads + nkv;
        const int h = is_q ? head : head - a.n_q_heads - (is_k ? 0 : nkv);
        const uint16_t *src = (const uint16_t *)(is_q ? a.q : is_k ? a.k : a.v) + h * D + v * 8;
        const long long step = is_q ? a.q_stride : is_k ? a.k_stride : a.v_stride;
        uint16_t *rows = (uint16_t *)(is_q ? a.q_out : is_k ? a.k_out : nullptr);
        const long long rows_step = is_q ? a.q_out_stride : a.k_out_stride;
        if (rows) rows += h * D + v * 8;
        uint16_t *cache = is_q ? nullptr : (uint16_t *)(is_k ? a.kv.k : a.kv.v) + (long long)h * ps * D + v * 8;
        uint4 x[TB], y[TB];
#pragma unroll
        for (int i = 0; i < TB; ++i)
            if (place[i].ok) {
                x[i] = *reinterpret_cast<const uint4 *>(src + (t0 + i) * step);
                y[i] = *reinterpret_cast<const uint4 *>(src + (t0 + i) * step + kHalf);
            }
#pragma unroll
        for (int i = 0; i < TB; ++i) {
            if (!place[i].ok) continue;
            if (is_q || is_k) rotate<T>(x[i], y[i], &cs[i][v * 8]);
            if (rows) {
                uint16_t *dst = rows + (t0 + i) * rows_step;
                *reinterpret_cast<uint4 *>(dst) = x[i];
                *reinterpret_cast<uint4 *>(dst + kHalf) = y[i];
            }
            if (cache) {
                uint16_t *dst = cache + place[i].row;
                *reinterpret_cast<uint4 *>(dst) = x[i];
                *reinterpret_cast<uint4 *>(dst + kHalf) = y[i];
            }
        }
    }
}

template <class T, int D>
void go(const AppendParams &p, int num_sms, cudaStream_t stream) {
    // One token a block up to four blocks an SM, then two (8192 tokens of
    // 32/8/128 heads: one 43.7 us, two 41.8, four 41.5, eight 49.8; 1300 ragged
    // ones: 9.5, 7.9, 8.4, 9.8; 16: 3.2, 3.4, 3.9, 5.2).
    const int n = p.a.n_tokens;
    if (n <= 4 * num_sms) kv_append_kernel<T, D, 1><<<n, kAppendThreads, 0, stream>>>(p);
    else kv_append_kernel<T, D, 2><<<n / 2 + n % 2, kAppendThreads, 0, stream>>>(p);
}

}  // namespace

cudaError_t append_launch(const AppendArgs &a, int num_sms, cudaStream_t stream) {
    AppendParams p;
    p.a = a;
    const int half = a.kv.head_dim / 2;
    // theta^(-2i/d) as powers of theta^(-2/d): the relative error grows by
    // 2^-53 a step, at most 64 of them
    const double step = pow((double)a.theta, -1.0 / half);
    double f = 1.0 / 6.283185307179586476925286766559;
    for (int i = 0; i < half; ++i, f *= step) p.turn[i] = f;
    if (a.kv.dtype == MK_BF16) {
        if (a.kv.head_dim == 64) go<Bf16, 64>(p, num_sms, stream);
        else go<Bf16, 128>(p, num_sms, stream);
    } else {
        if (a.kv.head_dim == 64) go<Fp16, 64>(p, num_sms, stream);
        else go<Fp16, 128>(p, num_sms, stream);
    }
    return cudaGetLastError();
}

}  // namespace mk
