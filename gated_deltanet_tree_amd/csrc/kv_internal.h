// Host side of the 4-bit cache calls, shared by their translation units: argument checks and the
// split of an attention call over workgroups.  Plain C++17, no HIP types.
#pragma once

#include "gdn_internal.h"

namespace gdn {

// Sizes, offsets and the pointers every cache call reads (pools, page table, lengths, offsets).
// `empty` is set when there is nothing to do.
gdn_status check_kv_args(const gdn_kv_args *a, const int32_t *host_seq_offsets, const char *who,
                         bool need_offsets, bool &empty);
// Heads and the launch's size of an attention call whose other sizes are checked.
gdn_status check_attention_sizes(const gdn_kv_args *a, const int32_t *host_seq_offsets, const char *who);
gdn_status check_aligned16(const void *const *ptrs, int n, const char *who, const char *names);

inline int log2_exact(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

// How an attention call is launched (see attention_work.h).
struct AttentionPlan {
    int32_t tile_rows;    // 32 or 64 rows (token x query head of one kv head) a workgroup walks with
    int32_t row_blocks;   // blocks of tile_rows in the longest sequence
    int32_t max_rows;     // rows of the largest block
    int32_t parts;        // equal parts a unit, a workgroup each; 0: the line is cut into shares
    int64_t units;        // of the launch: row_blocks a head, some of them empty in a ragged batch
    int64_t workgroups;   // parts of all units, or shares
    int64_t workspace;    // bytes: two fragments a workgroup, and where each unit's are
};
constexpr int64_t kCutBytes = 8;
AttentionPlan plan_attention(const gdn_kv_args *a, const int32_t *host_seq_offsets);
// The launch, and the join's of a workgroup twice as large, stay within the largest grid.
inline bool plan_fits(const AttentionPlan &p) { return p.workgroups <= kMaxBlocks && p.units <= kMaxBlocks / 2; }

}  // namespace gdn
