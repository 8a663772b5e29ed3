// Argument checks and work splits of the 4-bit cache and its attention (host, no device work).
#include <algorithm>

#include "kv_internal.h"

namespace gdn {

gdn_status check_aligned16(const void *const *ptrs, int n, const char *who, const char *names) {
    for (int i = 0; i < n; ++i) {
        if (ptrs[i] == nullptr) return fail(GDN_EINVAL, "%s: null pointer among %s", who, names);
        if (reinterpret_cast<uintptr_t>(ptrs[i]) % 16 != 0)
            return fail(GDN_EINVAL, "%s: %s must be 16-byte aligned", who, names);
    }
    return GDN_OK;
}

gdn_status check_kv_args(const gdn_kv_args *a, const int32_t *host_seq_offsets, const char *who,
                         bool need_offsets, bool &empty) {
    empty = true;
    if (a == nullptr || host_seq_offsets == nullptr)
        return fail(GDN_EINVAL, "%s: null arguments", who);
    if (a->n_seqs < 0 || a->n_seqs > kMaxSeqs || a->n_kv_heads < 1 || a->n_layers < 1 ||
        a->layer_begin < 0 || a->n_tokens < 0)
        return fail(GDN_EINVAL, "%s: bad n_seqs/n_kv_heads/n_layers/layer_begin/n_tokens", who);
    if (a->head_dim != 64 && a->head_dim != 128 && a->head_dim != 256)
        return fail(GDN_EINVAL, "%s: head_dim %d, only 64, 128 and 256 are supported", who,
                    a->head_dim);
    if (a->in_dtype != GDN_F32 && a->in_dtype != GDN_BF16)
        return fail(GDN_EINVAL, "%s: in_dtype %d", who, a->in_dtype);
    const int32_t pt = a->page_tokens;
    if (pt != 16 && pt != 32 && pt != 64 && pt != 128 && pt != 256)
        return fail(GDN_EINVAL, "%s: page_tokens %d, must be 16, 32, 64, 128 or 256", who, pt);
    if (a->n_pages < 1 || a->max_pages < 1)
        return fail(GDN_EINVAL, "%s: n_pages and max_pages must be >= 1", who);
    if (int64_t(a->max_pages) * pt > (int64_t(1) << 30))
        return fail(GDN_EINVAL, "%s: more than 2^30 slots a sequence", who);
    if (host_seq_offsets[0] != 0 || host_seq_offsets[a->n_seqs] != a->n_tokens)
        return fail(GDN_EINVAL, "%s: seq_offsets must run from 0 to n_tokens", who);
    for (int32_t b = 0; b < a->n_seqs; ++b)
        if (host_seq_offsets[b + 1] < host_seq_offsets[b])
            return fail(GDN_EINVAL, "%s: seq_offsets must not decrease (sequence %d)", who, b);
    if (a->n_seqs == 0) return GDN_OK;
    if (!a->pages || !a->length || (need_offsets && !a->seq_offsets))
        return fail(GDN_EINVAL, "%s: null pages/length/seq_offsets", who);
    const void *pools[] = {a->k_codes, a->v_codes, a->k_scales, a->v_scales};
    gdn_status st = check_aligned16(pools, 4, who, "k_codes/v_codes/k_scales/v_scales");
    if (st != GDN_OK) return st;
    empty = a->n_tokens == 0;
    return GDN_OK;
}

// Waves the device holds at two per SIMD.  A call whose row tiles alone reach that many runs each
// tile over all its tokens, four tiles to a workgroup; a smaller one is cut along the tokens until
// it does, but not below two 32-token tiles a wave.
constexpr int64_t kWaves = 2048;

AttentionPlan plan_attention(const gdn_kv_args *a, const int32_t *host_seq_offsets) {
    AttentionPlan p{};
    const int64_t group = a->n_heads / a->n_kv_heads;
    int64_t longest = 0;
    for (int32_t b = 0; b < a->n_seqs; ++b)
        longest = std::max<int64_t>(longest, host_seq_offsets[b + 1] - host_seq_offsets[b]);
    const bool wide = a->in_dtype == GDN_BF16 && a->head_dim <= 128 && longest * group > 32;
    p.tile_rows = wide ? 64 : 32;
    int64_t tiles = 0;
    for (int32_t b = 0; b < a->n_seqs; ++b) {
        const int64_t rows = (host_seq_offsets[b + 1] - host_seq_offsets[b]) * group;
        tiles += (rows + p.tile_rows - 1) / p.tile_rows;
    }
    tiles *= int64_t(a->n_kv_heads) * a->n_layers;
    const int64_t cap = int64_t(a->max_pages) * a->page_tokens;
    const int64_t len = a->max_length > 0 ? std::min<int64_t>(a->max_length, cap) : cap;
    p.row_groups = 1;
    p.splits = 1;
    if (tiles >= kWaves) {
        // fp32 rows hold three planes of q: four row groups of 256 channels pass the LDS
        p.row_groups = a->in_dtype == GDN_F32 && a->head_dim == 256 ? 1 : 4;
    } else if (tiles > 0) {
        const int64_t want = (kWaves / 4 + tiles - 1) / tiles;
        p.splits = int32_t(std::max<int64_t>(1, std::min<int64_t>(want, len / 256)));
    }
    const int64_t block_rows = int64_t(p.tile_rows) * p.row_groups;
    p.row_blocks = int32_t((longest * group + block_rows - 1) / block_rows);
    p.n_blocks = int64_t(p.row_blocks) * p.splits * a->n_seqs * a->n_kv_heads * a->n_layers;
    // partial outputs and their (max, sum) pairs
    p.workspace = p.splits == 1 ? 0
                                : int64_t(p.splits) * a->n_layers * a->n_tokens * a->n_heads *
                                      (a->head_dim + 2) * int64_t(sizeof(float));
    return p;
}

}  // namespace gdn

using namespace gdn;

extern "C" size_t gdn_attention_workspace_bytes(const gdn_kv_args *a,
                                                const int32_t *host_seq_offsets) {
    clear_error();
    if (a == nullptr || host_seq_offsets == nullptr || a->n_seqs < 1 || a->n_seqs > kMaxSeqs ||
        a->n_kv_heads < 1 || a->n_heads < 1 || a->n_heads % a->n_kv_heads != 0 ||
        a->n_layers < 1 || a->page_tokens < 1 || a->max_pages < 1 || a->n_tokens < 1)
        return 0;
    return size_t(plan_attention(a, host_seq_offsets).workspace);
}
