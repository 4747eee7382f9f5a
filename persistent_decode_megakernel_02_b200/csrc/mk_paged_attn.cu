// mk_paged_attn.cu -- attention of one new token per sequence over a paged
// cache.
//
// One block per (sequence, KV head): its warps take the positions in turn,
// scoring the KV head's query heads against each key, with a running maximum
// and sum per warp and head; the warps' states are merged at the end.
#include "mk_ops.cuh"

namespace mk {
namespace {

constexpr int kPagedWarps = 8;

template <class T, int D>
__global__ void __launch_bounds__(kPagedWarps * 32) paged_attn_kernel(PagedArgs a) {
    constexpr int E = D / 32;   // elements of a head per lane (consecutive)
    __shared__ float so[kPagedWarps][MK_MAX_GROUP][D];
    __shared__ float sm[kPagedWarps][MK_MAX_GROUP], sl[kPagedWarps][MK_MAX_GROUP];
    const int nkv = a.kv.n_kv_heads, G = a.n_q_heads / nkv, ps = a.kv.page_size;
    const int s = blockIdx.x / nkv, h = blockIdx.x % nkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int len = a.lens[s];
    if (len < 0 || len > a.max_len) {
        if (threadIdx.x == 0) bad_value(a.status);
        len = min(max(len, 0), a.max_len);
    }
    float q[MK_MAX_GROUP][E], o[MK_MAX_GROUP][E], m[MK_MAX_GROUP], l[MK_MAX_GROUP];
    for (int g = 0; g < MK_MAX_GROUP; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.f;
        for (int e = 0; e < E; ++e) {
            o[g][e] = 0.f;
            q[g][e] = 0.f;
        }
        if (g < G)
            for (int e = 0; e < E; e += 2) {
                const uint32_t w = *reinterpret_cast<const uint32_t *>((const uint16_t *)a.q + s * a.q_stride +
                                                                       (long long)(h * G + g) * D + lane * E + e);
                const float2 f = T::unpack(w);
                q[g][e] = f.x * a.scale;
                q[g][e + 1] = f.y * a.scale;
            }
    }
    for (int j = warp; j < len; j += kPagedWarps) {
        const int page = a.kv.page_table[(long long)s * a.kv.pages_per_seq + j / ps];
        if (page < 0 || page >= a.kv.num_pages) {
            if (lane == 0) bad_value(a.status);
            continue;
        }
        const long long at = (((long long)page * nkv + h) * ps + j % ps) * D + lane * E;
        float k[E], v[E];
        for (int e = 0; e < E; e += 2) {
            const float2 fk = T::unpack(*reinterpret_cast<const uint32_t *>((const uint16_t *)a.kv.k + at + e));
            const float2 fv = T::unpack(*reinterpret_cast<const uint32_t *>((const uint16_t *)a.kv.v + at + e));
            k[e] = fk.x; k[e + 1] = fk.y;
            v[e] = fv.x; v[e + 1] = fv.y;
        }
#pragma unroll
        for (int g = 0; g < MK_MAX_GROUP; ++g) {
            if (g >= G) break;
            float x = 0.f;
            for (int e = 0; e < E; ++e) x = fmaf(q[g][e], k[e], x);
            x = warp_sum(x);
            const float mn = fmaxf(m[g], x);
            const float c = mn == -INFINITY ? 1.f : __expf(m[g] - mn), w = x == -INFINITY ? 0.f : __expf(x - mn);
            m[g] = mn;
            l[g] = l[g] * c + w;
            for (int e = 0; e < E; ++e) o[g][e] = o[g][e] * c + w * v[e];
        }
    }
    for (int g = 0; g < G; ++g) {
        for (int e = 0; e < E; ++e) so[warp][g][lane * E + e] = o[g][e];
        if (lane == 0) { sm[warp][g] = m[g]; sl[warp][g] = l[g]; }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G * D / 2; i += blockDim.x) {
        const int g = i / (D / 2), e = i % (D / 2) * 2;
        float M = -INFINITY, L = 0.f, x = 0.f, y = 0.f;
        for (int w = 0; w < kPagedWarps; ++w) M = fmaxf(M, sm[w][g]);
        for (int w = 0; w < kPagedWarps; ++w) {
            const float c = sl[w][g] == 0.f ? 0.f : __expf(sm[w][g] - M);
            L += c * sl[w][g];
            x += c * so[w][g][e];
            y += c * so[w][g][e + 1];
        }
        const float r = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
        *reinterpret_cast<uint32_t *>((uint16_t *)a.out + s * a.out_stride + (long long)(h * G + g) * D + e) =
            T::pack(x * r, y * r);
    }
}

}  // namespace

size_t paged_workspace(const mk_paged_kv &, int, int, int) { return 0; }

cudaError_t paged_launch(const PagedArgs &a, int, int, cudaStream_t stream) {
    const int grid = a.kv.n_seqs * a.kv.n_kv_heads;
    if (a.kv.dtype == MK_BF16) {
        if (a.kv.head_dim == 64) paged_attn_kernel<Bf16, 64><<<grid, kPagedWarps * 32, 0, stream>>>(a);
        else paged_attn_kernel<Bf16, 128><<<grid, kPagedWarps * 32, 0, stream>>>(a);
    } else {
        if (a.kv.head_dim == 64) paged_attn_kernel<Fp16, 64><<<grid, kPagedWarps * 32, 0, stream>>>(a);
        else paged_attn_kernel<Fp16, 128><<<grid, kPagedWarps * 32, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace mk
