// Driver of the fragments' bookkeeping for the sanitized host build: what the workgroups of an
// attention call write (the first share of every unit, a fragment a run) against what the join reads,
// over lengths far below the expected one, which cost less than the parts they are cut into.  Arrays
// are heap blocks of exactly the workspace's sizes.  Prints "ok" and exits 0.
#include <cstdio>
#include <vector>

#include "attention_work.h"
#include "kv_internal.h"

static int failures = 0;
static void expect(const char *what, bool ok) {
    if (!ok && ++failures < 20) std::printf("FAIL %s\n", what);
}

static void check_parts() {
    for (int64_t cost : {int64_t(1), int64_t(288), int64_t(298), int64_t(544), int64_t(767), int64_t(768), int64_t(1) << 40})
        for (int parts : {1, 2, 255, 384, 512, 768}) {
            int64_t at = 0;
            int begins = 0;
            for (int i = 0; i < parts; ++i) {
                const gdn::Run r = gdn::part_of(cost, i, parts);
                expect("parts follow on one another", r.x == at && r.length >= 0);
                begins += r.begins;
                expect("the first part begins the unit", r.begins == (i == 0));
                at += r.length;
            }
            expect("parts cover the unit", at == cost && begins == 1);
        }
}

// The equal-parts launch of a plan over device lengths `past`: every unit's runs, then the join.
static void check_plan(int d, int dtype, int kv_heads, int group, const std::vector<int> &news,
                       const std::vector<int> &past, int capacity, int max_length, bool tree) {
    gdn_kv_args a{};
    const int S = int(news.size());
    a.n_seqs = S;
    a.n_kv_heads = kv_heads;
    a.n_heads = kv_heads * group;
    a.head_dim = d;
    a.page_tokens = 64;
    a.max_pages = (capacity + 63) / 64;
    a.n_layers = 1;
    a.in_dtype = dtype;
    a.max_length = max_length;
    std::vector<int32_t> offs{0};
    for (int n : news) offs.push_back(offs.back() + n);
    a.n_tokens = offs.back();
    const gdn::AttentionPlan p = gdn::plan_attention(&a, offs.data());
    if (p.parts <= 1) return;
    std::vector<int> fragments(size_t(2 * p.workgroups), -1);  // the unit that wrote it
    std::vector<int> first(size_t(p.units), -1);
    for (int64_t share = p.workgroups - 1; share >= 0; --share) {  // any order: the last writer shows
        int64_t i = share;
        const int part = int(i % p.parts);
        i /= p.parts;
        const int64_t unit = i;
        const int block = int(i % p.row_blocks);
        const int seq = int(i / p.row_blocks / kv_heads % S);
        const gdn::SeqWork w = gdn::seq_work(past[seq], news[seq], group, p.tile_rows, tree, int64_t(a.max_pages) * 64);
        if (block >= w.blocks) continue;
        const gdn::Run r = gdn::part_of(w.a + w.b * block, part, p.parts);
        int &slot = fragments.at(size_t(gdn::fragment_at(share, r.begins)));
        expect("a fragment is written once", slot == -1);
        slot = int(unit);
        if (r.begins) {
            expect("one share begins a unit", first[size_t(unit)] == -1);
            first[size_t(unit)] = int(share);
        }
    }
    for (int64_t unit = 0; unit < p.units; ++unit) {
        if (first[size_t(unit)] < 0) continue;
        for (int f = 0; f < p.parts; ++f) {
            const int64_t at = gdn::fragment_at(first[size_t(unit)] + f, f == 0);
            expect("the join reads what the unit wrote", at < int64_t(fragments.size()) && fragments[size_t(at)] == unit);
        }
    }
}

int main() {
    check_parts();
    for (int d : {64, 128, 256})
        for (int dtype : {GDN_F32, GDN_BF16})
            for (int heads : {1, 2, 3})
                for (int group : {1, 2, 5})
                    for (int len : {0, 1, 10, 50, 479, 480, 100000})
                        for (int capacity : {4096, 73728, 131072, 262144, 1 << 20})
                            for (bool tree : {false, true}) {
                                check_plan(d, dtype, heads, group, {1}, {len}, capacity, 0, tree);
                                check_plan(d, dtype, heads, group, {9}, {len}, capacity, capacity / 2, tree);
                                check_plan(d, dtype, heads, group, {1, 1}, {len, 100000}, 262144, 100001, tree);
                                check_plan(d, dtype, heads, group, {1, 0, 3}, {len, 200000, 5}, capacity, 0, tree);
                            }
    if (failures) return 1;
    std::printf("ok\n");
    return 0;
}
