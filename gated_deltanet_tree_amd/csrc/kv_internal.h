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
AttentionPlan plan_attention(const gdn_kv_args *a, const int32_t *host_seq_offsets,
                             const gdn_sparse_args *sparse = nullptr);
// The launch, and the join's of a workgroup twice as large, stay within the largest grid.
inline bool plan_fits(const AttentionPlan &p) { return p.workgroups <= kMaxBlocks && p.units <= kMaxBlocks / 2; }

// Sparse attention: what the selection and the attention check beyond check_attention_sizes, the
// selections of the longest sequence, and how the selection is launched.
constexpr int32_t kMaxTopPages = 256;
gdn_status check_sparse_sizes(const gdn_kv_args *a, const gdn_sparse_args *s, const int32_t *host_seq_offsets,
                              const char *who);
int64_t sparse_selections(const gdn_kv_args *a, const gdn_sparse_args *s, const int32_t *host_seq_offsets);

constexpr int32_t kSparePages = 64;   // pages kept beside the best where it is not sure yet which those are
constexpr int32_t kJoinPages = 2048;  // best pages joined at once
struct SelectPlan {
    int64_t selections;  // of the longest sequence: units a sequence and head, some of them empty
    int64_t units;
    int64_t row_tiles;   // 16 rows each, of the largest selection
    int32_t splits;
    bool narrow;         // workgroups of 8 waves, two a compute unit, not of 16
    int32_t room;        // pages a share hands to the join: all of its own, or its best
    int64_t workspace;
};
SelectPlan plan_select(const gdn_kv_args *a, const gdn_sparse_args *s, const int32_t *host_seq_offsets);
// Its workgroups are four times as large as the largest grid is counted in.
inline bool select_fits(const SelectPlan &p) { return p.units * p.splits <= kMaxBlocks / 4; }

}  // namespace gdn
