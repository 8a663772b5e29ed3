// Driver of the sparse attention's work split for the sanitized host build: rows of selections in blocks,
// slots of a selection, and what the workgroups of a launch write (equal parts of units, or shares of the
// work line) against what the join reads.  Arrays are heap blocks of exactly the workspace's sizes.
// Prints "ok" and exits 0.
#include <algorithm>
#include <climits>
#include <cstdio>
#include <vector>

#include "attention_work.h"
#include "kv_internal.h"

static int failures = 0;
static void expect(const char *what, bool ok) {
    if (!ok && ++failures < 20) std::printf("FAIL %s\n", what);
}

// Every row of a sequence is in exactly one block, of its own selection, and every block holds rows.
static void check_rows(int n_new, int share, int group, int tile, bool tree) {
    const gdn::SparseShape x{4, share};
    const gdn::SeqWork w = gdn::sparse_work(x, 1000, n_new, group, tile, tree, 4096, 4);
    const int tokens = share == 0 || share > n_new ? n_new : share;
    std::vector<int> seen(size_t(n_new) * group, 0);
    for (int k = 0; k < int(w.blocks); ++k) {
        const gdn::SparseRows r = gdn::sparse_rows(x, k, n_new, group, tile);
        expect("a block holds rows", r.first < r.end);
        expect("and no more than a tile", r.end - r.first <= tile);
        expect("of one selection", r.token % tokens == 0 && r.first >= r.token * group &&
                                       r.end <= std::min(r.token + tokens, n_new) * group);
        for (int i = r.first; i < r.end; ++i) ++seen.at(size_t(i));
    }
    expect("every row once", std::all_of(seen.begin(), seen.end(), [](int c) { return c == 1; }));
    // a launch has blocks for the longest sequence: those past a sequence's own hold none
    for (int k = int(w.blocks); k < int(w.blocks) + 40; ++k) {
        const gdn::SparseRows r = gdn::sparse_rows(x, k, n_new, group, tile);
        expect("no rows behind the last block", r.first >= r.end);
    }
    int64_t cost = 0;
    for (int64_t k = 0; k < w.blocks; ++k) {
        expect("a block costs something", w.a + w.b * k > 0);
        expect("a block's place on the line", gdn::cost_before(w, k) == cost);
        expect("and back", gdn::block_at(w, cost) == k && gdn::block_at(w, cost + w.a + w.b * k - 1) == k);
        cost += w.a + w.b * k;
    }
    expect("the sequence's cost", cost == w.cost);
}

static void check_slots() {
    for (int shift : {4, 6, 8})
        for (int top : {1, 7, 256})
            for (int64_t capacity : {int64_t(256), int64_t(65536), int64_t(1) << 30})
                for (int64_t length : {int64_t(INT_MIN), int64_t(-1), int64_t(0), int64_t(1), int64_t(255), int64_t(256),
                                       int64_t(65537), int64_t(INT_MAX)}) {
                    const int past = gdn::length_of(length, capacity);
                    const gdn::SparseSlots s = gdn::sparse_slots({top, 1}, past, capacity, shift);
                    expect("full pages", s.full == past >> shift && s.chosen == std::min(s.full, top));
                    expect("slots of the pages taken, then the tail", s.past == (s.chosen << shift) + past % (1 << shift));
                    expect("slots left out", capacity - s.capacity == int64_t(s.full - s.chosen) << shift);
                }
}

struct Shape {
    int d, dtype, kv_heads, group, page, max_pages, top, share, max_length, layers;
    bool tree;
    std::vector<int> news, past;
};

static int lines, parts;

static void check_plan(const Shape &c) {
    gdn_kv_args a{};
    const int S = int(c.news.size());
    a.n_seqs = S;
    a.n_kv_heads = c.kv_heads;
    a.n_heads = c.kv_heads * c.group;
    a.head_dim = c.d;
    a.n_pages = 4;
    a.page_tokens = c.page;
    a.max_pages = c.max_pages;
    a.n_layers = c.layers;
    a.in_dtype = c.dtype;
    a.max_length = c.max_length;
    std::vector<int32_t> offs{0};
    for (int n : c.news) offs.push_back(offs.back() + n);
    a.n_tokens = offs.back();
    gdn_sparse_args s{};
    s.top_pages = c.top;
    s.share_tokens = c.share;
    expect("sizes", gdn::check_sparse_sizes(&a, &s, offs.data(), "driver") == GDN_OK);
    const gdn::AttentionPlan p = gdn::plan_attention(&a, offs.data(), &s);
    expect("the query's size covers the plan", int64_t(gdn_sparse_workspace_bytes(&a, &s, offs.data())) >= p.workspace);
    int shift = 0;
    while (1 << shift < c.page) ++shift;
    const gdn::SparseShape x{c.top, c.share};
    const int64_t capacity = int64_t(c.max_pages) << shift;
    std::vector<gdn::SeqWork> work;
    int64_t most = 0;
    for (int b = 0; b < S; ++b) {
        work.push_back(gdn::sparse_work(x, c.past[b], c.news[b], c.group, p.tile_rows, c.tree, capacity, shift));
        most = std::max(most, work.back().blocks);
    }
    expect("a launch has the blocks of its longest sequence", p.row_blocks == most);
    if (p.parts == 1) return;
    struct Cut {
        int64_t first = -1, count = 0;
    };
    std::vector<Cut> cut(size_t(p.units), Cut{});
    std::vector<int64_t> fragments(size_t(2 * p.workgroups), -1);  // the unit that wrote it
    std::vector<int64_t> end(size_t(p.units), 0);                   // the tile its runs have come to
    std::vector<int> runs(size_t(p.units), 0);
    auto unit_of = [&](int li, int seq, int head, int64_t block) {
        return ((int64_t(li) * S + seq) * c.kv_heads + head) * p.row_blocks + block;
    };
    // [x, x1) of a unit by workgroup `share`
    auto walk = [&](int64_t share, int li, int seq, int head, int64_t block, int64_t x0, int64_t x1, bool begins, int64_t count) {
        const int64_t unit = unit_of(li, seq, head, block), cost = work[size_t(seq)].a + work[size_t(seq)].b * block;
        const gdn::SparseSlots at = gdn::sparse_slots(x, gdn::length_of(c.past[size_t(seq)], capacity), capacity, shift);
        const gdn::SparseRows r = gdn::sparse_rows(x, int(block), c.news[size_t(seq)], c.group, p.tile_rows);
        const int last = c.tree ? c.news[size_t(seq)] - 1 : (r.end - 1) / c.group;
        const int tiles = (gdn::slots_upto(at.past, last, at.capacity) + 31) / 32;
        const int t0 = gdn::tile_at(x0, cost, tiles), t1 = gdn::tile_at(x1, cost, tiles);
        expect("tiles follow on one another", t0 == end[size_t(unit)] && t1 >= t0);
        end[size_t(unit)] = t1;
        if (x1 == cost) expect("to the last", t1 == tiles);
        ++runs[size_t(unit)];
        if (begins) {
            expect("a unit begins once", cut[size_t(unit)].first == -1);
            cut[size_t(unit)] = {share, count};
        }
        if (p.parts == 0 && x0 == 0 && x1 == cost) return;  // written whole
        int64_t &slot = fragments.at(size_t(gdn::fragment_at(share, begins)));
        expect("a fragment is written once", slot == -1);
        slot = unit;
    };
    if (p.parts != 0) {
        ++parts;
        for (int li = 0; li < c.layers; ++li)
            for (int b = 0; b < S; ++b)
                for (int64_t block = 0; block < work[size_t(b)].blocks; ++block)
                    for (int head = 0; head < c.kv_heads; ++head)
                        for (int part = 0; part < p.parts; ++part) {
                            const gdn::SeqWork &w = work[size_t(b)];
                            // as a launch numbers them: parts, heads, blocks from the last, sequences, layers
                            const int64_t share = (((int64_t(li) * S + b) * p.row_blocks + p.row_blocks - 1 - block) * c.kv_heads + head) * p.parts + part;
                            const gdn::Run r = gdn::part_of(w.a + w.b * block, part, p.parts);
                            walk(share, li, b, head, block, r.x, r.x + r.length, r.begins, p.parts);
                        }
    } else {
        ++lines;
        int64_t total = 0;
        for (const gdn::SeqWork &w : work) total += w.cost * c.kv_heads;
        total *= c.layers;
        const int64_t q = (total + p.workgroups - 1) / p.workgroups;
        int64_t at = 0;
        for (int li = 0; li < c.layers; ++li)
            for (int b = 0; b < S; ++b)
                for (int head = 0; head < c.kv_heads; ++head)
                    for (int64_t block = 0; block < work[size_t(b)].blocks; ++block) {
                        const int64_t cost = work[size_t(b)].a + work[size_t(b)].b * block;
                        for (int64_t x0 = 0; x0 < cost;) {
                            const int64_t share = (at + x0) / q, x1 = std::min(cost, (share + 1) * q - at);
                            expect("a share of the launch", share < p.workgroups);
                            const int64_t count = x1 < cost ? 1 + gdn::quotient(cost - x1 + q - 1, q) : 1;
                            walk(share, li, b, head, block, x0, x1, x0 == 0, count);
                            x0 = x1;
                        }
                        at += cost;
                    }
        expect("the line", at == total);
    }
    for (int64_t unit = 0; unit < p.units; ++unit) {
        const Cut &u = cut[size_t(unit)];
        if (u.first < 0) continue;
        expect("as many runs as the join is told", runs[size_t(unit)] == u.count);
        if (u.count == 1) continue;
        for (int64_t f = 0; f < u.count; ++f)
            expect("the join reads what the unit wrote", fragments.at(size_t(gdn::fragment_at(u.first + f, f == 0))) == unit);
    }
}

// The largest launch of the selection is accepted, the next larger one is not.
static void check_grid() {
    const int n = 1 << 20;
    const std::vector<int32_t> offs{0, n};
    gdn_kv_args a{};
    a.n_seqs = a.n_heads = a.n_kv_heads = 1;
    a.head_dim = 128;
    a.n_tokens = n;
    a.n_pages = a.max_pages = 4;
    a.page_tokens = 64;
    a.in_dtype = GDN_BF16;
    gdn_sparse_args s{};
    s.top_pages = 2;
    s.share_tokens = 1;
    for (int layers : {1, 3, 4, 7}) {
        a.n_layers = layers;
        expect("sizes", gdn::check_sparse_sizes(&a, &s, offs.data(), "driver") == GDN_OK);
        const gdn::SelectPlan p = gdn::plan_select(&a, &s, offs.data());
        expect("a selection a token", p.units == int64_t(layers) * n && p.splits == 1);
        expect("workgroups of up to 1024 threads, fewer than 2^32 in all", gdn::select_fits(p) == (int64_t(layers) * n * 1024 < int64_t(1) << 32));
    }
}

int main() {
    for (int tile : {32, 64})
        for (int group : {1, 3, 4, 16, 20})
            for (int share : {0, 1, 3, 16, 64, 1000})
                for (int n : {1, 2, 16, 17, 33, 64, 65, 130, 193, 777}) check_rows(n, share, group, tile, false);
    for (int tile : {32, 64})
        for (int group : {1, 6, 20})
            for (int n : {1, 22, 64}) check_rows(n, 0, group, tile, true);
    check_slots();
    check_grid();
    const std::vector<int> shorts(14, 1), longs{9000, 8600, 100, 900, 30, 0, 2000, 64, 63, 700, 128, 1500, 3000, 5};
    for (int d : {64, 128, 256})
        for (int dtype : {GDN_F32, GDN_BF16})
            for (int heads : {1, 2, 4})
                for (int group : {1, 4, 6, 16})
                    for (int top : {20, 52, 128, 256}) {
                        for (int layers : {1, 3}) {
                            const Shape base{d, dtype, heads, group, 64, 160, top, 1, 0, layers, false, {}, {}};
                            auto with = [&](int share, bool tree, std::vector<int> news, std::vector<int> past, int len) {
                                Shape c = base;
                                c.share = share;
                                c.tree = tree;
                                c.news = news;
                                c.past = past;
                                c.max_length = len;
                                check_plan(c);
                            };
                            with(1, false, shorts, longs, 0);
                            with(16, false, {700, 130, 1, 77}, {5000, 3700, 200, 4000}, 0);
                            with(64, false, {193, 65, 70, 3, 0}, {9500, 6500, 6000, 300, 7}, 0);
                            with(63, false, {190, 64, 1}, {INT_MAX, -5, 60}, 5000);
                            with(0, false, {300, 2, 0, 65}, {100, 9000, 50, 8000}, 0);
                            with(0, true, {22, 1, 64, 0, 33, 22}, {9000, 10, 8500, 3, 4000, 70}, 0);
                            with(0, true, std::vector<int>(14, 22), longs, 0);
                            with(0, true, {22}, {9000}, 0);
                            with(1, false, {1}, {9000}, 0);
                        }
                    }
    expect("parts and lines are reached", parts > 100 && lines > 100);
    if (failures) return 1;
    std::printf("ok\n");
    return 0;
}
