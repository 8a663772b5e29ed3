// Argument checks and work splits of the 4-bit cache and its attention (host, no device work).
#include <algorithm>

#include "attention_work.h"
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

static gdn_status check_kv_sizes(const gdn_kv_args *a, const int32_t *host_seq_offsets, const char *who) {
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
    return GDN_OK;
}

gdn_status check_kv_args(const gdn_kv_args *a, const int32_t *host_seq_offsets, const char *who,
                         bool need_offsets, bool &empty) {
    empty = true;
    gdn_status st = check_kv_sizes(a, host_seq_offsets, who);
    if (st != GDN_OK) return st;
    if (a->n_seqs == 0) return GDN_OK;
    if (!a->pages || !a->length || (need_offsets && !a->seq_offsets))
        return fail(GDN_EINVAL, "%s: null pages/length/seq_offsets", who);
    const void *pools[] = {a->k_codes, a->v_codes, a->k_scales, a->v_scales};
    st = check_aligned16(pools, 4, who, "k_codes/v_codes/k_scales/v_scales");
    if (st != GDN_OK) return st;
    empty = a->n_tokens == 0;
    return GDN_OK;
}

gdn_status check_attention_sizes(const gdn_kv_args *a, const int32_t *host_seq_offsets, const char *who) {
    if (a->n_heads < 1 || a->n_heads % a->n_kv_heads != 0)
        return fail(GDN_EINVAL, "%s: n_heads must be a multiple of n_kv_heads", who);
    if (int64_t(a->n_tokens) * a->n_heads > INT32_MAX)
        return fail(GDN_EINVAL, "%s: more than 2^31 rows", who);
    if (a->n_tokens >= 1 << 30)  // a capacity and a token's number add up in 31 bits
        return fail(GDN_EINVAL, "%s: 2^30 tokens or more", who);
    // in blocks of 32 rows, as many as the plan's units or twice as many: keeps its products small
    int64_t longest = 0;
    for (int32_t b = 0; b < a->n_seqs; ++b)
        longest = std::max<int64_t>(longest, host_seq_offsets[b + 1] - host_seq_offsets[b]);
    const int64_t blocks = (longest * (a->n_heads / a->n_kv_heads) + 31) / 32 * a->n_seqs;
    const int64_t heads = int64_t(a->n_kv_heads) * a->n_layers;
    if (blocks > 0 && heads > kMaxBlocks / blocks)
        return fail(GDN_EINVAL, "%s: too many workgroups", who);
    return GDN_OK;
}

// Blocks of tile_rows rows that the sequences of a sparse call have, and those of the longest.
static void sparse_blocks(const gdn_kv_args *a, const gdn_sparse_args *s, const int32_t *host_seq_offsets,
                          int64_t tile_rows, int64_t &all, int64_t &most) {
    const int64_t group = a->n_heads / a->n_kv_heads;
    all = most = 0;
    for (int32_t b = 0; b < a->n_seqs; ++b) {
        const int64_t n = host_seq_offsets[b + 1] - host_seq_offsets[b];
        if (n == 0) continue;
        const int64_t blocks = sparse_blocks(SparseShape{s->top_pages, s->share_tokens}, int(n), group, tile_rows);
        all += blocks;
        most = std::max(most, blocks);
    }
}

int64_t sparse_selections(const gdn_kv_args *a, const gdn_sparse_args *s, const int32_t *host_seq_offsets) {
    int64_t most = 0;
    for (int32_t b = 0; b < a->n_seqs; ++b) {
        const int64_t n = host_seq_offsets[b + 1] - host_seq_offsets[b];
        if (n == 0) continue;
        const int64_t tokens = sparse_tokens(SparseShape{s->top_pages, s->share_tokens}, int(n));
        most = std::max(most, (n + tokens - 1) / tokens);
    }
    return most;
}

gdn_status check_sparse_sizes(const gdn_kv_args *a, const gdn_sparse_args *s, const int32_t *host_seq_offsets,
                              const char *who) {
    if (s->top_pages < 1 || s->top_pages > kMaxTopPages)
        return fail(GDN_EINVAL, "%s: top_pages %d, must be 1 to %d", who, s->top_pages, kMaxTopPages);
    if (s->keep_first < 0 || s->keep_last < 0 || int64_t(s->keep_first) + s->keep_last > s->top_pages)
        return fail(GDN_EINVAL, "%s: keep_first %d and keep_last %d of top_pages %d", who, s->keep_first,
                    s->keep_last, s->top_pages);
    if (s->share_tokens < 0) return fail(GDN_EINVAL, "%s: share_tokens must not be negative", who);
    if (int64_t(a->n_tokens) * a->n_heads > 1 << 30)  // block and row numbers past the end stay in 31 bits
        return fail(GDN_EINVAL, "%s: more than 2^30 rows", who);
    // a selection has a block at least, however few its rows
    int64_t all, most;
    sparse_blocks(a, s, host_seq_offsets, 32, all, most);
    const int64_t heads = int64_t(a->n_kv_heads) * a->n_layers, blocks = most * a->n_seqs;
    if (blocks > 0 && heads > kMaxBlocks / 2 / blocks) return fail(GDN_EINVAL, "%s: too many workgroups", who);
    return GDN_OK;
}

// Workgroups of four waves the device's 256 CUs hold: two a CU by the registers, three with 64
// channels and one row tile.
constexpr int64_t kCus = 256;
// A unit is not cut into parts of less than kMinTiles tiles of 32 slots (two a wave), nor at all
// up to kWholeTiles: joining the pieces would cost more than it saves.  us a call, whole / cut, at 18,
// 25 and 32 tiles: one token, 16 / 4 heads of 64, 8.3 / 10.6, 9.4 / 10.6, 10.0 / 10.4; a tree of 22
// nodes, 48 / 8 heads of 128, 16.6 / 18.9, 17.8 / 18.2, 18.9 / 17.5; at 18, 28 and 32: 32 tokens,
// 16 / 2 heads of 128 in fp32, 11.1 / 12.8, 13.2 / 13.4, 14.3 / 12.9; one token, 16 / 2 heads of 256,
// 14.2 / 15.1, 16.5 / 15.8, 17.6 / 14.8, and in fp32, the one form that would rather be cut from 24 on,
// 16.6 / 16.9, 19.6 / 17.3, 21.3 / 16.0.
// The line of shares pays where units differ in length and a workgroup has more than kLineTiles to
// walk; below, finding its place on the line and starting a second unit there takes longer than the
// uneven end.
// With many units a workgroup takes one whole and the hardware deals them: no fragments to write and
// join, and the workgroups of a sequence run together and share its pages in L2.  From how many units
// a slot on that is ahead, in halves (us whole / line, lengths spread over a factor of 4 to 8):
//   kEven, bf16 with two row tiles a wave or 64 channels: trees of 22 nodes, 48 / 8 heads of 128,
//   235 / 197 at 1.0, 279 / 294 at 1.5, 501 / 537 at 3, 719 / 790 at 4.5; 32 / 8 heads of 64, one token,
//   99 / 108 at 1.3, 145 / 155 at 2, 324 / 347 at 5.3, and six, 106 / 114 at 1.5, 190 / 210 at 3;
//   kEvenTile, bf16 with one row tile of more than 16 rows: trees of 13 nodes, 16 / 8 heads of 128,
//   131 / 130 at 1.5, 154 / 163 at 2, 224 / 232 at 3; trees of 22, 16 / 2 heads of 256, 169 / 164 at 1.5,
//   210 / 206 at 2, 312 / 328 at 3; 64 tokens, 8 heads of 256, 224 / 283 at 2, 330 / 423 at 3;
//   kEvenMemory, bound by memory, or by the three planes of fp32: one token, heads of 128, 86 / 82 at
//   1, 163 / 159 at 2, 273 / 276 at 4, 407 / 410 at 6; 16 / 2 heads of 256, 571 / 523 at 2, 803 / 769 at 3,
//   1058 / 1032 at 4; fp32 trees of 22, 16 / 4 heads of 64, 172 / 158 at 1.5, 219 / 199 at 2, 397 / 416 at 4,
//   of 128, 252 / 226 at 2, 350 / 353 at 3, 473 / 487 at 4, and 16 / 2 of 256, 447 / 398 at 2, 622 / 614 at 3,
//   835 / 843 at 4.
// A launch has units for the longest sequence's blocks in every sequence.  Where one sequence has
// most of the rows, parts for the units that exist would be mostly empty workgroups, with room for
// their fragments (100 sequences of 1 token and one of 800, 8 / 1 heads of 128: 20000 of them and 1.3
// GB), so beyond kSpread workgroups a slot the parts are as few as all the units leave, and a line
// where those would hold more than kPartTiles tiles (us a call, parts / line, of such batches with
// 2 to 40 sequences: up to 63 tiles a part 30.5 / 37.5, 27.7 / 35.4, 23.7 / 30.9, 36.4 / 31.8; 66 to 99 tiles
// 25.9 / 32.5, 50.6 / 38.4, 36.8 / 42.2, 35.2 / 47.0, 26.7 / 31.3; from 103 on 52.8 / 37.6, 51.1 / 37.1, 58.6 /
// 38.1; the batch above 57.4 / 56.9 at 119, and 83.9 in parts for the units that exist).
// Sparse calls go by the same rule, though a selection's pages and a tail are nearly as long in every unit, so that
// the line has less to even out.  us of the attention and its join, by the rule / whole / two parts / line, and the units
// that have rows:
//   trees of 22 nodes, 48 / 8 heads of 128, 67 pages of 64: 96 units (rule: five parts) 36.3 / 48.7 / 37.2 / 42.1, 192
//   (line) 52.0 / 49.6 / 50.0 / 51.8, 384 (line) 78.4 / 73.6 / 86.7 / 78.5, 768 (whole) 130 / 131 / 135 / 134; in fp32, 320
//   (line) 76.6 / 87.9 / 81.4 / 76.1; 24 / 4 heads of 256, 160 (three parts) 42.6 / 48.8 / 51.4 / 51.3;
//   one token, 32 / 8 heads of 128, 35 pages: 128 (four parts) 19.3 / 22.5 / 19.4 / 26.9, 256 (two parts) 24.9 / 23.5 /
//   24.9 / 32.1, 512 (line) 45.0 / 32.9 / 42.4 / 45.2;
//   chunks of prompts, 16 tokens a selection, 32 / 8 heads of 128, 35 pages: 360 (line) 56.6 / 44.8 / 53.7 / 56.9, 696
//   (line) 88.1 / 69.7 / 90.9 / 87.9, 1224 (whole) 110 / 110 / 149 / 134; in fp32, 1368 (line) 162 / 153 / 171 / 162.
// Where the rule takes the line for bf16 rows, whole units would be ahead from a third of a unit a slot on.
constexpr int64_t kMinTiles = 8, kWholeTiles = 28, kLineTiles = 48, kEven = 3, kEvenTile = 4, kEvenMemory = 8;
constexpr int64_t kSpread = 2, kPartTiles = 96;

AttentionPlan plan_attention(const gdn_kv_args *a, const int32_t *host_seq_offsets, const gdn_sparse_args *sparse) {
    AttentionPlan p{};
    const int64_t group = a->n_heads / a->n_kv_heads;
    int64_t longest = 0;
    for (int32_t b = 0; b < a->n_seqs; ++b)
        longest = std::max<int64_t>(longest, host_seq_offsets[b + 1] - host_seq_offsets[b]);
    const int64_t cap = int64_t(a->max_pages) * a->page_tokens;
    int64_t len = a->max_length > 0 ? std::min<int64_t>(a->max_length, cap) : cap;
    if (sparse != nullptr) {  // the slots of a selection, a page begun, and the new tokens'
        len = std::min(len, int64_t(sparse->top_pages + 1) * a->page_tokens + longest);
        if (sparse->share_tokens != 0) longest = std::min<int64_t>(longest, sparse->share_tokens);
    }
    // Two row tiles a wave share the work of unpacking the keys and values; fp32 rows and 256
    // channels leave registers for one.
    const bool bf16 = a->in_dtype == GDN_BF16;
    const bool wide = bf16 && a->head_dim <= 128 && longest * group > 32;
    p.tile_rows = wide ? 64 : 32;
    p.max_rows = int32_t(std::min<int64_t>(p.tile_rows, longest * group));
    p.row_blocks = int32_t((longest * group + p.tile_rows - 1) / p.tile_rows);
    int64_t blocks = 0;
    for (int32_t b = 0; b < a->n_seqs; ++b)
        blocks += ((host_seq_offsets[b + 1] - host_seq_offsets[b]) * group + p.tile_rows - 1) / p.tile_rows;
    if (sparse != nullptr) {
        int64_t most;
        sparse_blocks(a, sparse, host_seq_offsets, p.tile_rows, blocks, most);
        p.row_blocks = int32_t(most);
    }
    const int64_t heads = int64_t(a->n_kv_heads) * a->n_layers;
    const int64_t tiles = (len + 31) / 32;  // of the longest unit expected
    const int64_t slots = kCus * (!wide && a->head_dim == 64 ? 3 : 2);
    p.units = int64_t(p.row_blocks) * a->n_seqs * heads;
    const int64_t even = !bf16 || (a->head_dim > 64 && longest * group <= 16) ? kEvenMemory
                         : wide || a->head_dim == 64                            ? kEven
                                                                                : kEvenTile;
    if (tiles <= kWholeTiles || 2 * blocks * heads >= even * slots) {
        p.parts = 1;  // enough units that the hardware's own dealing evens them out
    } else if (blocks * heads * tiles <= kLineTiles * slots ||
               (a->n_seqs == 1 && p.row_blocks == 1 && heads <= slots)) {
        p.parts = int32_t(std::max<int64_t>(1, std::min(slots / (blocks * heads), tiles / kMinTiles)));
        if (p.parts > 1 && p.units * p.parts > kSpread * slots) {
            p.parts = int32_t(std::max<int64_t>(1, std::min(slots / p.units, tiles / kMinTiles)));
            if (tiles > kPartTiles * p.parts) p.parts = 0;
        }
    }
    p.workgroups = p.parts != 0 ? p.units * p.parts : slots;
    p.workspace = p.parts == 1 ? 0
                               : p.units * kCutBytes + p.workgroups * 2 * p.tile_rows * (a->head_dim + 2) *
                                                           int64_t(sizeof(float));
    return p;
}

// Splits of a selection's pages: none up to kWholeBytes of limits to read (a compute unit gets 35 GB/s of them)
// and kWholeTurns tiles of 16 pages and 16 rows for every wave, as a join takes 9 us and more; beyond, shares of
// kSplitBytes or kSplitTurns, no more workgroups than the device has compute units, and no more best pages in all
// than the join holds at once.  Shares hand on all their pages if the join can hold them, else their best.
// us, whole / in shares: one token, 16 heads of 64, 20000 slots in pages of 32 (160 KB), 15.5 / 16.5; trees of 22
// nodes, 48 heads, 8 caches of up to 65000 slots (520 KB), 43 / 35; 2 caches of 262000 slots, 256 channels (2.1
// MB), 73 / 25.
// More selections than compute units are taken two a compute unit, by workgroups of half as many waves: one waits
// while the other computes.  us a call of selection and attention, 16 waves / 8: 40 tokens, 32 / 8 heads of 128,
// up to 5000 slots 54 / 45, 40000 slots 65 / 55, 100000 slots 87 / 86, in fp32 74 / 65; chunks of prompts, 16 tokens a
// selection, 131 / 117.
constexpr int64_t kWholeBytes = 256 * 1024, kWholeTurns = 64, kSplitBytes = 128 * 1024, kSplitTurns = 16;

SelectPlan plan_select(const gdn_kv_args *a, const gdn_sparse_args *s, const int32_t *host_seq_offsets) {
    SelectPlan p{};
    p.selections = sparse_selections(a, s, host_seq_offsets);
    p.units = p.selections * a->n_seqs * a->n_kv_heads * a->n_layers;
    const int64_t cap = int64_t(a->max_pages) * a->page_tokens;
    const int64_t len = a->max_length > 0 ? std::min<int64_t>(a->max_length, cap) : cap;
    const int64_t pages = len / a->page_tokens;
    int64_t tokens = 0;
    for (int32_t b = 0; b < a->n_seqs; ++b)
        tokens = std::max<int64_t>(tokens, host_seq_offsets[b + 1] - host_seq_offsets[b]);
    if (s->share_tokens != 0) tokens = std::min<int64_t>(tokens, s->share_tokens);
    p.row_tiles = (tokens * (a->n_heads / a->n_kv_heads) + 15) / 16;
    const int64_t bytes = pages * 4 * a->head_dim, turns = (pages + 15) / 16 * p.row_tiles / 16;
    const int64_t work = bytes <= kWholeBytes && turns <= kWholeTurns ? 1 : std::max(bytes / kSplitBytes, turns / kSplitTurns);
    const int64_t want = p.units > 0 ? (kCus + p.units - 1) / p.units : 1, best = s->top_pages + kSparePages;
    p.splits = int32_t(std::max<int64_t>(1, std::min({want, work, kJoinPages / best})));
    p.narrow = p.units > kCus;  // then no splits either
    p.room = int32_t(std::max(best, (std::min<int64_t>(pages, kJoinPages) + p.splits - 1) / p.splits));
    // pages' scores and table entries, a share's count and error
    p.workspace = p.splits == 1 ? 0 : p.units * p.splits * 8 * (p.room + 1);
    return p;
}

}  // namespace gdn

using namespace gdn;

extern "C" size_t gdn_attention_workspace_bytes(const gdn_kv_args *a,
                                                const int32_t *host_seq_offsets) {
    clear_error();
    const char *who = "gdn_attention_workspace_bytes";
    if (check_kv_sizes(a, host_seq_offsets, who) != GDN_OK || a->n_tokens == 0 ||
        check_attention_sizes(a, host_seq_offsets, who) != GDN_OK)
        return 0;
    const AttentionPlan plan = plan_attention(a, host_seq_offsets);
    return plan_fits(plan) ? size_t(plan.workspace) : 0;
}

extern "C" size_t gdn_sparse_workspace_bytes(const gdn_kv_args *a, const gdn_sparse_args *s,
                                             const int32_t *host_seq_offsets) {
    clear_error();
    const char *who = "gdn_sparse_workspace_bytes";
    if (s == nullptr) {
        fail(GDN_EINVAL, "%s: null arguments", who);
        return 0;
    }
    if (check_kv_sizes(a, host_seq_offsets, who) != GDN_OK || a->n_tokens == 0 ||
        check_attention_sizes(a, host_seq_offsets, who) != GDN_OK ||
        check_sparse_sizes(a, s, host_seq_offsets, who) != GDN_OK)
        return 0;
    const AttentionPlan plan = plan_attention(a, host_seq_offsets, s);
    const SelectPlan select = plan_select(a, s, host_seq_offsets);
    return plan_fits(plan) && select_fits(select) ? size_t(std::max(plan.workspace, select.workspace)) : 0;
}
