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
// their angle, then one 32-bit sincospi.  Then each thread moves 16-byte
// pairs of vectors (elements i.. and i + d/2..) of a head through registers.
#include "mk_ops.cuh"

namespace mk {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendMaxTokens = 8;   // tokens per block, at most (one lookup per warp)

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

template <class T, int D>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ AppendParams p, int tb) {
    constexpr int kHalf = D / 2, kVecs = kHalf / 8;   // 16-byte vectors in half a head
    __shared__ float2 cs[kAppendMaxTokens][kHalf];
    __shared__ Place place[kAppendMaxTokens];
    const AppendArgs &a = p.a;
    const long long t0 = (long long)blockIdx.x * tb;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nkv = a.kv.n_kv_heads, ps = a.kv.page_size;

    for (int i = warp; i < tb; i += kAppendThreads / 32) {
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

    // one item: vector v of head h of token i; heads are q, then k, then v
    const int heads = a.n_q_heads + 2 * nkv, per_token = heads * kVecs;
    for (int it = threadIdx.x; it < tb * per_token; it += kAppendThreads) {
        const int i = it / per_token, r = it - i * per_token;
        if (!place[i].ok) continue;
        const int head = r / kVecs, v = r % kVecs;
        const long long t = t0 + i;
        const uint16_t *src;
        if (head < a.n_q_heads) src = (const uint16_t *)a.q + t * a.q_stride + head * D;
        else if (head < a.n_q_heads + nkv) src = (const uint16_t *)a.k + t * a.k_stride + (head - a.n_q_heads) * D;
        else src = (const uint16_t *)a.v + t * a.v_stride + (head - a.n_q_heads - nkv) * D;
        uint4 x = *reinterpret_cast<const uint4 *>(src + v * 8);
        uint4 y = *reinterpret_cast<const uint4 *>(src + v * 8 + kHalf);
        if (head < a.n_q_heads + nkv) rotate<T>(x, y, &cs[i][v * 8]);
        if (head < a.n_q_heads) {
            uint16_t *dst = (uint16_t *)a.q_out + t * a.q_out_stride + head * D + v * 8;
            *reinterpret_cast<uint4 *>(dst) = x;
            *reinterpret_cast<uint4 *>(dst + kHalf) = y;
            continue;
        }
        const bool is_k = head < a.n_q_heads + nkv;
        const int h = head - a.n_q_heads - (is_k ? 0 : nkv);
        if (is_k && a.k_out) {
            uint16_t *dst = (uint16_t *)a.k_out + t * a.k_out_stride + h * D + v * 8;
            *reinterpret_cast<uint4 *>(dst) = x;
            *reinterpret_cast<uint4 *>(dst + kHalf) = y;
        }
        uint16_t *dst = (uint16_t *)(is_k ? a.kv.k : a.kv.v) + place[i].row + (long long)h * ps * D + v * 8;
        *reinterpret_cast<uint4 *>(dst) = x;
        *reinterpret_cast<uint4 *>(dst + kHalf) = y;
    }
}

}  // namespace

cudaError_t append_launch(const AppendArgs &a, cudaStream_t stream) {
    AppendParams p;
    p.a = a;
    const int half = a.kv.head_dim / 2;
    // theta^(-2i/d) as powers of theta^(-2/d): the relative error grows by
    // 2^-53 a step, at most 64 of them
    const double step = pow((double)a.theta, -1.0 / half);
    double f = 1.0 / 6.283185307179586476925286766559;
    for (int i = 0; i < half; ++i, f *= step) p.turn[i] = f;
    const int tb = 1;
    const int grid = (a.n_tokens + tb - 1) / tb;
    if (a.kv.dtype == MK_BF16) {
        if (a.kv.head_dim == 64) kv_append_kernel<Bf16, 64><<<grid, kAppendThreads, 0, stream>>>(p, tb);
        else kv_append_kernel<Bf16, 128><<<grid, kAppendThreads, 0, stream>>>(p, tb);
    } else {
        if (a.kv.head_dim == 64) kv_append_kernel<Fp16, 64><<<grid, kAppendThreads, 0, stream>>>(p, tb);
        else kv_append_kernel<Fp16, 128><<<grid, kAppendThreads, 0, stream>>>(p, tb);
    }
    return cudaGetLastError();
}

}  // namespace mk
