// mk_kv_append.cu -- append rotated keys and values to a paged cache.
//
// For every new token: q' = R(pos) q, k' = R(pos) k with the half-split
// rotation of the decode step, k' and v into the cache row of the token's
// position.  Per token it reads (nq + 2 nkv) d elements and writes (nq +
// 2 nkv) d (and nkv d more with k_out), 3 flops each: bound by memory.
//
// A block takes one token.  Its warps look up the token's sequence and
// check its place; then the block fills a table of cos / sin in shared
// memory, one angle per pair: pos * theta^(-2i/d) / (2 pi) in 64 bits with the
// whole turns dropped, so that positions of any size keep their angle, then
// one 32-bit sincospi.  Then a thread takes a 16-byte pair of vectors (elements
// i.. and i + d/2..) of one head at a time.  Nothing but the angles passes
// between threads, and enough blocks are resident to hide the look-up: 8192
// tokens of 32/8/128 heads take 37.3 us, 221 MB at 89 % of the copy rate.
#include "mk_ops.cuh"

namespace mk {
namespace {

struct AppendParams {
    AppendArgs a;
    double turn[64];   // theta^(-2i/d) / (2 pi)
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

template <class T, int D, int NT>
__global__ void __launch_bounds__(NT) kv_append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int kHalf = D / 2, kVecs = kHalf / 8;   // 16-byte vectors in half a head
    __shared__ float2 cs[kHalf];
    const AppendArgs &a = p.a;
    const int t = blockIdx.x, lane = threadIdx.x & 31;
    const int nkv = a.kv.n_kv_heads, ps = a.kv.page_size, ns = a.kv.n_seqs;
    // every warp for itself: the look-ups of one block hit the same lines
    if (t >= a.cu[ns]) return;
    const int s = warp_find_seq(a.cu, ns, t);
    const int first = a.cu[s];
    const long long pos = (long long)a.start[s] + t - first;
    bool ok = first >= 0 && t >= first && t < a.cu[s + 1] && pos >= 0 && pos < (long long)a.kv.pages_per_seq * ps;
    long long row = 0;     // element offset of (page, head 0, row) in the cache
    if (ok) {
        const int page = a.kv.page_table[(long long)s * a.kv.pages_per_seq + (int)pos / ps];
        ok = page >= 0 && page < a.kv.num_pages;
        row = ((long long)page * nkv * ps + (int)pos % ps) * D;
    }
    if (!ok) {
        if (threadIdx.x == 0) bad_value(a.status);
        return;
    }
    for (int j = threadIdx.x; j < kHalf; j += NT) {
        const double turns = (double)pos * p.turn[j];
        float sn, cn;
        sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cn);
        cs[j] = make_float2(cn, sn);
    }
    __syncthreads();

    // vector v of a head; heads are q, then k, then v
    const int heads = a.n_q_heads + 2 * nkv;
#pragma unroll 1
    for (int r = threadIdx.x; r < heads * kVecs; r += NT) {
        const int head = r / kVecs, v = r % kVecs;
        const bool is_q = head < a.n_q_heads, is_k = !is_q && head < a.n_q_heads + nkv;
        const int h = is_q ? head : head - a.n_q_heads - (is_k ? 0 : nkv);
        const int at = h * D + v * 8;
        const uint16_t *src = (const uint16_t *)(is_q ? a.q : is_k ? a.k : a.v) +
                              t * (is_q ? a.q_stride : is_k ? a.k_stride : a.v_stride) + at;
        uint4 x = *reinterpret_cast<const uint4 *>(src), y = *reinterpret_cast<const uint4 *>(src + kHalf);
        if (is_q || is_k) {
            rotate<T>(x, y, &cs[v * 8]);
            uint16_t *dst = (uint16_t *)(is_q ? a.q_out : a.k_out);
            if (dst) {
                dst += t * (is_q ? a.q_out_stride : a.k_out_stride) + at;
                *reinterpret_cast<uint4 *>(dst) = x;
                *reinterpret_cast<uint4 *>(dst + kHalf) = y;
            }
        }
        if (!is_q) {
            uint16_t *dst = (uint16_t *)(is_k ? a.kv.k : a.kv.v) + row + (long long)h * ps * D + v * 8;
            *reinterpret_cast<uint4 *>(dst) = x;
            *reinterpret_cast<uint4 *>(dst + kHalf) = y;
        }
    }
}

template <class T, int D>
cudaError_t go(const AppendParams &p, int num_sms, cudaStream_t stream) {
    // More threads a token while there are SMs to spare (32/8/128 heads, 256
    // and 128 threads: 16 tokens 3.4 and 3.7 us, 256 4.3 and 4.5, 512 5.2 and
    // 5.1, 8192 41.8 and 37.3; two tokens a block: 38.4, four: 40.9)
    const int n = p.a.n_tokens;
    return n <= 2 * num_sms ? launch_kernel(kv_append_kernel<T, D, 256>, n, 256, 0, stream, p)
                            : launch_kernel(kv_append_kernel<T, D, 128>, n, 128, 0, stream, p);
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
    if (a.kv.dtype == MK_BF16)
        return a.kv.head_dim == 64 ? go<Bf16, 64>(p, num_sms, stream) : go<Bf16, 128>(p, num_sms, stream);
    return a.kv.head_dim == 64 ? go<Fp16, 64>(p, num_sms, stream) : go<Fp16, 128>(p, num_sms, stream);
}

}  // namespace mk
