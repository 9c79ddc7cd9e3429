// Prompt-phase paged attention with a sliding window and first tokens that stay
// visible: the windowed form of the kernel in pkv_prefill.cuh, and its entry point.
#include "pkv_prefill.cuh"

using namespace pkv;

extern "C" pkv_status paged_attention_prefill_window(void *out, const void *query, const void *key_cache,
                                                     const void *value_cache, const int32_t *block_tables,
                                                     const int32_t *context_lens, const int32_t *query_start,
                                                     int num_seqs, int num_tokens, int max_query_len,
                                                     int max_blocks_per_seq, int block_size, int num_blocks,
                                                     int num_heads, int num_kv_heads, int head_dim, float scale,
                                                     int window, int num_sinks, void *workspace,
                                                     size_t workspace_bytes, pkv_dtype dtype,
                                                     struct CUstream_st *stream) {
    const char *what = "paged_attention_prefill_window";
    if (window < 1 || num_sinks < 0)
        return fail(PKV_EINVAL, "%s: window %d (at least 1), %d sinks (at least 0)", what, window, num_sinks);
    PrefillArgs a;
    const pkv_status rc = prefill_args(what, a, out, query, key_cache, value_cache, block_tables, context_lens, query_start,
                                       num_seqs, num_tokens, max_query_len, max_blocks_per_seq, block_size, num_blocks,
                                       num_heads, num_kv_heads, head_dim, scale, workspace, workspace_bytes, dtype);
    if (rc != PKV_OK || a.num_items == 0) return rc;
    // The kernel takes up to 96 + window from a row's place against a key tile, which goes down to -255: that stays
    // within 32 bits.  (Contexts of 2^31 - 1024 tokens and more, which would see less, fit no memory.  The same done
    // in the kernel, against its own limits, makes fp16 prompts 2.5 % slower.)
    a.window = window < INT_MAX - 1024 ? window : INT_MAX - 1024;
    a.sinks = num_sinks;
    a.sink_unit = num_sinks > 0 && (num_sinks & -num_sinks) < block_size ? num_sinks & -num_sinks : block_size;
    const cudaError_t e = launch_prefill<kWindow>(head_dim, dtype == PKV_BF16, a, query, key_cache, value_cache,
                                                  num_kv_heads, stream);
    if (e != cudaSuccess) return fail(PKV_ECUDA, "%s: launch: %s", what, cudaGetErrorString(e));
    return PKV_OK;
}
