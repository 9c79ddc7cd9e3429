// What the two halves of decode attention over shared prefixes hand to one
// another: the partial results of a prefix's partitions.
#pragma once

#include <cuda_runtime.h>

#include "pkv.h"

namespace pkv {

// Partition p of a prefix is its tokens [p * part, (p + 1) * part).  For every
// query row (sequence, head) the partition's scores' reference (log2 domain),
// the sum of 2^(score - reference) and the values' sum under those weights.
struct PrefixParts {
    float *m, *l;              // [S][H][slots]
    float *o;                  // [S][H][slots][D]
    int part;                  // tokens, a multiple of 128
    int max_parts;             // partitions of the longest prefix
    int own;                   // tokens of a partition of a sequence's own ones, where those go to memory too
    int slots;                 // of both
};

// Pairs of row tiles that groups may have after their first ones: `group` query
// heads per kv head, 128 rows to a tile.
inline int more_pairs(int num_seqs, int max_group_size, int group) {
    const int seqs = 2 * (128 / group);
    return max_group_size > seqs ? (num_seqs - 1) / seqs : 0;
}

// Its work items at most: beyond, looking for those with work could outlast the kernel's waits.
constexpr long long kMaxSharedItems = 1ll << 27;

// The prefix half over groups of many rows, on the fifth-generation tensor
// cores (shared_prefix.cu), on at most max_ctas SMs.  Arguments as checked by the
// caller.
cudaError_t launch_shared_prefix(const void *query, const void *key_cache, const void *value_cache,
                                 const int32_t *block_tables, const int32_t *context_lens,
                                 const int32_t *group_start, const int32_t *prefix_lens,
                                 int num_groups, int num_seqs, int max_group_size, int max_prefix, int max_blocks,
                                 int block_size, int num_blocks, int num_heads, int num_kv_heads, int head_dim,
                                 float scale_log2, const PrefixParts &parts, bool bf16, int max_ctas,
                                 cudaStream_t stream);

}  // namespace pkv
