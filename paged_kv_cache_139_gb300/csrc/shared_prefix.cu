// Decode over shared prefixes, its prefix half for groups of many rows: the shared
// form of the kernel in pkv_prefill.cuh.  Groups of few rows and the sequences' own
// tokens are in attention_span.cu, with the entry point.
#include "pkv_prefill.cuh"

namespace pkv {

cudaError_t launch_shared_prefix(const void *query, const void *key_cache, const void *value_cache,
                                 const int32_t *block_tables, const int32_t *context_lens,
                                 const int32_t *group_start, const int32_t *prefix_lens,
                                 int num_groups, int num_seqs, int max_group_size, int max_prefix, int max_blocks,
                                 int block_size, int num_blocks, int num_heads, int num_kv_heads, int head_dim,
                                 float scale_log2, const PrefixParts &parts, bool bf16, int max_ctas,
                                 cudaStream_t stream) {
    PrefillArgs a = {};
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.status = status_ptr();
    a.num_seqs = num_seqs;
    a.num_tokens = num_seqs;                       // of the query's tensor map: one row each
    a.max_blocks = max_blocks;
    a.log2_block = ilog2(block_size);
    a.num_blocks = num_blocks;
    a.num_heads = num_heads;
    a.group = num_heads / num_kv_heads;
    a.scale_log2 = scale_log2;
    a.group_start = group_start;
    a.prefix_lens = prefix_lens;
    a.num_groups = num_groups;
    a.max_group = max_group_size;
    a.max_prefix = max_prefix;
    a.num_kv_heads = num_kv_heads;
    a.tile_seqs = kRows / a.group;
    a.part_tiles = parts.part / kKeys;
    a.num_parts = parts.max_parts;
    a.parts = parts;
    a.num_pairs = more_pairs(num_seqs, max_group_size, a.group);
    a.num_items = (num_groups + a.num_pairs) * a.num_parts * num_kv_heads;   // (the caller has checked that it is one)
    if (!a.status) return cudaErrorInvalidValue;
    a.max_ctas = max_ctas;
    return launch_prefill<kShared>(head_dim, bf16, a, query, key_cache, value_cache, num_kv_heads, stream);
}

}  // namespace pkv
