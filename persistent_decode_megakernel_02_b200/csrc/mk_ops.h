// mk_ops.h -- host-side interface between the serving operators' C entry
// points (mk_ops.cpp: argument checks) and their launchers (mk_kv_append.cu,
// mk_paged_attn.cu, mk_prompt_attn.cu, mk_sample.cu).  Not part of the public
// ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/mk.h"

namespace mk {

constexpr int kOpsMaxDevices = 64;

struct AppendArgs {
    mk_paged_kv kv;
    const int32_t *cu, *start;
    int n_tokens, n_q_heads;
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    float theta;
    void *q_out, *k_out;
    long long q_out_stride, k_out_stride;
    int32_t *status;
};
cudaError_t append_launch(const AppendArgs &a, int num_sms, cudaStream_t stream);

struct PagedArgs {
    mk_paged_kv kv;
    const int32_t *lens;
    int max_len, n_q_heads;
    const void *q;
    void *out;
    long long q_stride, out_stride;
    float scale;
    void *workspace;
    int32_t *status;
};
size_t paged_workspace(const mk_paged_kv &kv, int max_len, int num_sms);
cudaError_t paged_launch(const PagedArgs &a, int num_sms, cudaStream_t stream);

struct PromptArgs {
    int dtype, nq, nkv, d;
    const int32_t *cu;
    int n_seqs, n_tokens, max_len;
    const void *q, *k, *v;
    void *out;
    long long q_stride, k_stride, v_stride, out_stride;
    float scale;
    int32_t *status;
};
// The guard's share of a tile of 128 values (rows of 64 elements, in the
// 128-byte swizzle; for 128 dims two halves one after the other): the 16-byte
// vector that a lane of guard warp `half` looks at in a step, d / 8 steps in
// all.  A warp's vectors hold the columns [half d / 2, + d / 2) of every row.
// (64 dims: half a row of eight rows a step, in an order in which eight lanes
// touch every bank once.)
__host__ __device__ constexpr int guard_vector(int d, int half, int step, int lane) {
    return d == 128 ? half * 1024 + step * 32 + lane
                    : (step * 8 + (lane >> 3) + (lane & 4)) * 8 + ((((lane >> 2) & 1) ^ half) << 2 | (lane & 3));
}
// row and first column of a vector
__host__ __device__ constexpr int guard_row(int vec) { return vec / 8 % 128; }
__host__ __device__ constexpr int guard_column(int vec) { return vec / 1024 * 64 + ((vec ^ guard_row(vec)) & 7) * 8; }

cudaError_t prompt_launch(const PromptArgs &a, int device, int num_sms, cudaStream_t stream);

struct SampleArgs {
    const float *logits;
    long long stride;
    int rows, vocab;
    const float *uniform, *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p;
    int32_t *token;
};
cudaError_t sample_launch(const SampleArgs &a, int device, int num_sms, cudaStream_t stream);

}  // namespace mk
