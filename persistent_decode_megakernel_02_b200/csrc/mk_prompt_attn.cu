// mk_prompt_attn.cu -- causal attention over packed prompts with grouped
// heads.
//
// One warp per (token, query head) walks the sequence's keys up to its own
// with a running maximum and sum.
#include "mk_ops.cuh"

namespace mk {
namespace {

template <class T, int D>
__global__ void __launch_bounds__(256) prompt_attn_kernel(PromptArgs a) {
    constexpr int E = D / 32;
    const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < a.n_seqs; i += blockDim.x) {
            const int b = a.cu[i], e = a.cu[i + 1];
            if (b < 0 || e < b || e > a.n_tokens || e - b > a.max_len) bad_value(a.status);
        }
    if (item >= (long long)a.n_tokens * a.nq) return;
    const int t = (int)(item / a.nq), hq = (int)(item % a.nq), h = hq / (a.nq / a.nkv);
    if (t >= a.cu[a.n_seqs]) return;
    const int s = warp_find_seq(a.cu, a.n_seqs, t);
    const int b = a.cu[s], e1 = a.cu[s + 1];
    if (b < 0 || b > t || e1 <= t || e1 > a.n_tokens || e1 - b > a.max_len) return;
    float q[E], o[E], m = -INFINITY, l = 0.f;
    for (int e = 0; e < E; e += 2) {
        const float2 f = T::unpack(*reinterpret_cast<const uint32_t *>((const uint16_t *)a.q + t * a.q_stride +
                                                                       (long long)hq * D + lane * E + e));
        q[e] = f.x * a.scale; q[e + 1] = f.y * a.scale;
        o[e] = o[e + 1] = 0.f;
    }
    for (int j = b; j <= t; ++j) {
        float x = 0.f, v[E];
        for (int e = 0; e < E; e += 2) {
            const float2 f = T::unpack(*reinterpret_cast<const uint32_t *>((const uint16_t *)a.k + j * a.k_stride +
                                                                           (long long)h * D + lane * E + e));
            const float2 g = T::unpack(*reinterpret_cast<const uint32_t *>((const uint16_t *)a.v + j * a.v_stride +
                                                                           (long long)h * D + lane * E + e));
            x = fmaf(q[e], f.x, fmaf(q[e + 1], f.y, x));
            v[e] = g.x; v[e + 1] = g.y;
        }
        x = warp_sum(x);
        const float mn = fmaxf(m, x);
        const float c = mn == -INFINITY ? 1.f : __expf(m - mn), w = x == -INFINITY ? 0.f : __expf(x - mn);
        m = mn;
        l = l * c + w;
        for (int e = 0; e < E; ++e) o[e] = o[e] * c + w * v[e];
    }
    const float r = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t *>((uint16_t *)a.out + t * a.out_stride + (long long)hq * D + lane * E + e) =
            T::pack(o[e] * r, o[e + 1] * r);
}

}  // namespace

cudaError_t prompt_launch(const PromptArgs &a, int, int, cudaStream_t stream) {
    const long long grid = ((long long)a.n_tokens * a.nq + 7) / 8;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (a.dtype == MK_BF16) {
        if (a.d == 64) prompt_attn_kernel<Bf16, 64><<<(int)grid, 256, 0, stream>>>(a);
        else prompt_attn_kernel<Bf16, 128><<<(int)grid, 256, 0, stream>>>(a);
    } else {
        if (a.d == 64) prompt_attn_kernel<Fp16, 64><<<(int)grid, 256, 0, stream>>>(a);
        else prompt_attn_kernel<Fp16, 128><<<(int)grid, 256, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace mk
