// Prompt-phase (prefill) paged attention: the causal form of the kernel in
// pkv_prefill.cuh, and its entry point.
#include "pkv_prefill.cuh"

namespace pkv {

long long prefill_items(int num_seqs, int num_tokens, int max_query_len, int num_heads, int num_kv_heads) {
    const bool head_pairs = pairs_heads(num_heads, num_kv_heads);
    return row_pairs(num_tokens, max_query_len, head_pairs) * (head_pairs ? num_heads / 2 : num_heads) * num_seqs;
}

}  // namespace pkv

using namespace pkv;

extern "C" pkv_status paged_attention_prefill(void *out, const void *query, const void *key_cache,
                                              const void *value_cache, const int32_t *block_tables,
                                              const int32_t *context_lens, const int32_t *query_start, int num_seqs,
                                              int num_tokens, int max_query_len, int max_blocks_per_seq,
                                              int block_size, int num_blocks, int num_heads, int num_kv_heads,
                                              int head_dim, float scale, void *workspace, size_t workspace_bytes,
                                              pkv_dtype dtype, struct CUstream_st *stream) {
    PrefillArgs a;
    const pkv_status rc = prefill_args("paged_attention_prefill", a, out, query, key_cache, value_cache, block_tables,
                                       context_lens, query_start, num_seqs, num_tokens, max_query_len,
                                       max_blocks_per_seq, block_size, num_blocks, num_heads, num_kv_heads, head_dim,
                                       scale, workspace, workspace_bytes, dtype);
    if (rc != PKV_OK || a.num_items == 0) return rc;
    const cudaError_t e = launch_prefill<kCausal>(head_dim, dtype == PKV_BF16, a, query, key_cache, value_cache,
                                                  num_kv_heads, stream);
    if (e != cudaSuccess) return fail(PKV_ECUDA, "paged_attention_prefill: launch: %s", cudaGetErrorString(e));
    return PKV_OK;
}
