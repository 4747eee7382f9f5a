// mk_ops.cpp -- C entry points of the serving operators (include/mk.h): every
// argument the host can see is checked here, before anything touches the
// device; the kernels and their launch rules are in mk_kv_append.cu,
// mk_paged_attn.cu, mk_prompt_attn.cu and mk_sample.cu.
#include <atomic>
#include <cmath>

#include "mk_ops.h"

using namespace mk;

namespace {

bool aligned(const void *p, uintptr_t n) { return p && ((uintptr_t)p & (n - 1)) == 0; }
bool aligned_or_null(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// rows of 16-bit elements: pointer and stride as the header asks
bool rows_ok(const void *p, long long stride, long long width) {
    return aligned(p, 16) && stride >= width && stride % 8 == 0;
}

bool heads_ok(int nq, int nkv, int d, int dtype) {
    return nkv >= 1 && nkv <= (1 << 16) && nq >= 1 && nq % nkv == 0 && nq / nkv <= MK_MAX_GROUP &&
           (d == 64 || d == 128) && (dtype == MK_BF16 || dtype == MK_FP16);
}

// sizes of a paged cache; every position fits an int
bool cache_sizes_ok(const mk_paged_kv *kv) {
    return kv && kv->n_seqs >= 1 && kv->pages_per_seq >= 1 && kv->num_pages >= 1 && kv->page_size >= 1 &&
           kv->n_kv_heads >= 1 && kv->n_kv_heads <= (1 << 16) && (kv->head_dim == 64 || kv->head_dim == 128) &&
           (kv->dtype == MK_BF16 || kv->dtype == MK_FP16) &&
           (long long)kv->pages_per_seq * kv->page_size <= 0x7fffff00LL &&
           // rows of the cache fit an int (more would not fit the device)
           (double)kv->num_pages * kv->n_kv_heads * kv->page_size <= 2147483647.0;
}

bool cache_ok(const mk_paged_kv *kv) {
    return cache_sizes_ok(kv) && aligned(kv->k, 16) && aligned(kv->v, 16) && aligned(kv->page_table, 4);
}

// The current device and its SM count; the properties are looked up once per
// device.
int ops_device(int *dev_out, int *sms_out) {
    static std::atomic<int> sms[kOpsMaxDevices];   // 0: not looked up, -1: unsupported
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return MK_ERR_CUDA;
    }
    if (dev < 0 || dev >= kOpsMaxDevices) return MK_ERR_INVALID;
    int n = sms[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        int major = 0, minor = 0, count = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            return MK_ERR_CUDA;
        }
        n = major == 10 && minor == 0 && count > 0 ? count : -1;
        sms[dev].store(n, std::memory_order_relaxed);
    }
    if (n < 0) return MK_ERR_INVALID;
    *dev_out = dev;
    *sms_out = n;
    return MK_OK;
}

// A failed launch leaves no sticky error behind for the caller's next CUDA
// call to trip over.
int launched(cudaError_t e) {
    if (e == cudaSuccess) return MK_OK;
    cudaGetLastError();
    return MK_ERR_CUDA;
}

}  // namespace

extern "C" {

int mk_kv_append(const mk_paged_kv *kv, const int32_t *cu_tokens, const int32_t *start_pos, int n_tokens,
                 int n_q_heads, const void *q, long long q_stride, const void *k, long long k_stride,
                 const void *v, long long v_stride, float rope_theta, void *q_out, long long q_out_stride,
                 void *k_out, long long k_out_stride, int32_t *status_out, mk_stream_t stream) {
    if (!cache_ok(kv) || !aligned(cu_tokens, 4) || !aligned(start_pos, 4) || !aligned_or_null(status_out, 4))
        return MK_ERR_INVALID;
    if (n_tokens < 0 || !(rope_theta > 1.f) || std::isinf(rope_theta)) return MK_ERR_INVALID;
    const long long kw = (long long)kv->n_kv_heads * kv->head_dim, qw = (long long)n_q_heads * kv->head_dim;
    if (n_q_heads == 0) {
        if (q || q_out) return MK_ERR_INVALID;
    } else {
        if (!heads_ok(n_q_heads, kv->n_kv_heads, kv->head_dim, kv->dtype)) return MK_ERR_INVALID;
        if (!rows_ok(q, q_stride, qw) || !rows_ok(q_out, q_out_stride, qw)) return MK_ERR_INVALID;
    }
    if (!rows_ok(k, k_stride, kw) || !rows_ok(v, v_stride, kw)) return MK_ERR_INVALID;
    if (k_out && !rows_ok(k_out, k_out_stride, kw)) return MK_ERR_INVALID;
    // an in-place output keeps its input's rows where they are
    if ((q_out == q && q && q_out_stride != q_stride) || (k_out == k && k_out_stride != k_stride)) return MK_ERR_INVALID;
    if (n_tokens == 0) return MK_OK;
    // rows that overlap in any other way, as far as the first elements tell
    if (q && (q_out == k || q_out == v || q_out == k_out || k_out == q)) return MK_ERR_INVALID;
    if (k_out && k_out == v) return MK_ERR_INVALID;
    int dev, sms;
    const int st = ops_device(&dev, &sms);
    if (st != MK_OK) return st;
    AppendArgs a{*kv, cu_tokens, start_pos, n_tokens, n_q_heads, q, k, v, q_stride, k_stride, v_stride, rope_theta,
                 q_out, k_out, q_out_stride, k_out_stride, status_out};
    return launched(append_launch(a, sms, (cudaStream_t)stream));
}

int mk_paged_attention_workspace(const mk_paged_kv *kv, int max_len, int n_q_heads, size_t *bytes_out) {
    if (!bytes_out) return MK_ERR_INVALID;
    *bytes_out = 0;
    if (!cache_sizes_ok(kv) || !heads_ok(n_q_heads, kv->n_kv_heads, kv->head_dim, kv->dtype)) return MK_ERR_INVALID;
    if (max_len < 0 || max_len > (long long)kv->pages_per_seq * kv->page_size) return MK_ERR_INVALID;
    int dev, sms;
    const int st = ops_device(&dev, &sms);
    if (st != MK_OK) return st;
    *bytes_out = paged_workspace(*kv, max_len, sms);
    return MK_OK;
}

int mk_paged_attention(const mk_paged_kv *kv, const int32_t *kv_lens, int max_len, int n_q_heads, const void *q,
                       long long q_stride, float scale, void *out, long long out_stride, void *workspace,
                       size_t workspace_bytes, int32_t *status_out, mk_stream_t stream) {
    if (!cache_ok(kv) || !aligned(kv_lens, 4) || !aligned_or_null(status_out, 4)) return MK_ERR_INVALID;
    if (!heads_ok(n_q_heads, kv->n_kv_heads, kv->head_dim, kv->dtype)) return MK_ERR_INVALID;
    if (max_len < 0 || max_len > (long long)kv->pages_per_seq * kv->page_size) return MK_ERR_INVALID;
    const long long qw = (long long)n_q_heads * kv->head_dim;
    if (!rows_ok(q, q_stride, qw) || !rows_ok(out, out_stride, qw)) return MK_ERR_INVALID;
    if (!(scale > 0.f) || std::isinf(scale)) return MK_ERR_INVALID;
    if (out == q && kv->n_seqs > 1 && out_stride != q_stride) return MK_ERR_INVALID;
    if (!aligned_or_null(workspace, 16)) return MK_ERR_INVALID;
    // the work, in steps of 16 positions and their overheads, fits an int
    if (((double)max_len / 16 + 32) * kv->n_seqs * kv->n_kv_heads > 2147000000.0) return MK_ERR_INVALID;
    int dev, sms;
    const int st = ops_device(&dev, &sms);
    if (st != MK_OK) return st;
    const size_t need = paged_workspace(*kv, max_len, sms);
    if (!workspace || workspace_bytes < need) return MK_ERR_INVALID;
    PagedArgs a{*kv, kv_lens, max_len, n_q_heads, q, out, q_stride, out_stride, scale, workspace, status_out};
    return launched(paged_launch(a, sms, (cudaStream_t)stream));
}

int mk_prompt_attention(int dtype, int n_q_heads, int n_kv_heads, int head_dim, const int32_t *cu_seqlens,
                        int n_seqs, int n_tokens, int max_len, const void *q, long long q_stride, const void *k,
                        long long k_stride, const void *v, long long v_stride, float scale, void *out,
                        long long out_stride, int32_t *status_out, mk_stream_t stream) {
    if (!heads_ok(n_q_heads, n_kv_heads, head_dim, dtype)) return MK_ERR_INVALID;
    if (!aligned(cu_seqlens, 4) || !aligned_or_null(status_out, 4)) return MK_ERR_INVALID;
    if (n_seqs < 1 || n_tokens < 0 || n_tokens > 0x7ffffc00 || max_len < 0) return MK_ERR_INVALID;
    // the (row block, head) items fit an int
    if (((double)n_tokens / 128 + n_seqs) * n_q_heads > 2147000000.0) return MK_ERR_INVALID;
    const long long qw = (long long)n_q_heads * head_dim, kw = (long long)n_kv_heads * head_dim;
    if (!rows_ok(q, q_stride, qw) || !rows_ok(out, out_stride, qw) || !rows_ok(k, k_stride, kw) ||
        !rows_ok(v, v_stride, kw))
        return MK_ERR_INVALID;
    if (!(scale > 0.f) || std::isinf(scale)) return MK_ERR_INVALID;
    if (n_tokens == 0) return MK_OK;
    if (out == k || out == v) return MK_ERR_INVALID;      // read by other blocks meanwhile
    int dev, sms;
    const int st = ops_device(&dev, &sms);
    if (st != MK_OK) return st;
    PromptArgs a{dtype, n_q_heads, n_kv_heads, head_dim, cu_seqlens, n_seqs, n_tokens, max_len, q, k, v, out, q_stride, k_stride, v_stride, out_stride,
                 scale, status_out};
    return launched(prompt_launch(a, dev, sms, (cudaStream_t)stream));
}

int mk_sample(const float *logits, long long row_stride, int rows, int vocab, const float *uniform,
              const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
              int32_t *token_out, mk_stream_t stream) {
    if (!aligned(logits, 4) || !aligned(uniform, 4) || !aligned(token_out, 4) || !aligned_or_null(temperature, 4) ||
        !aligned_or_null(top_k, 4) || !aligned_or_null(top_p, 4) || !aligned_or_null(min_p, 4))
        return MK_ERR_INVALID;
    if (rows < 0 || rows > (1 << 24) || vocab < 1 || vocab > MK_MAX_VOCAB || row_stride < vocab) return MK_ERR_INVALID;
    if (rows == 0) return MK_OK;
    int dev, sms;
    const int st = ops_device(&dev, &sms);
    if (st != MK_OK) return st;
    SampleArgs a{logits, row_stride, rows, vocab, uniform, temperature, top_k, top_p, min_p, token_out};
    return launched(sample_launch(a, dev, sms, (cudaStream_t)stream));
}

}  // extern "C"
