// Host side of the 4-bit cache calls, shared by their translation units: argument checks and the
// split of an attention call over workgroups.  Plain C++17, no HIP types.
#pragma once

#include "gdn_internal.h"

namespace gdn {

// Sizes, offsets and the pointers every cache call reads (pools, page table, lengths, offsets).
// `empty` is set when there is nothing to do.
gdn_status check_kv_args(const gdn_kv_args *a, const int32_t *host_seq_offsets, const char *who,
                         bool need_offsets, bool &empty);
gdn_status check_aligned16(const void *const *ptrs, int n, const char *who, const char *names);

inline int log2_exact(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

// How an attention call is cut: a workgroup of four waves holds row_groups waves of tile_rows rows
// each; the other 4 / row_groups waves of a row group, and `splits` workgroups, share its cached
// tokens.
struct AttentionPlan {
    int32_t tile_rows;   // 32 or 64 rows (token x query head of one kv head) a wave
    int32_t row_groups;  // 1 or 4
    int32_t splits;
    int32_t row_blocks;  // workgroups along the rows of the longest sequence
    int64_t n_blocks;
    int64_t workspace;   // bytes
};
AttentionPlan plan_attention(const gdn_kv_args *a, const int32_t *host_seq_offsets);

}  // namespace gdn
