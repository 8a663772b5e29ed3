// Driver of the attention's launch plans for the sanitized host build: the workspace query answers 0
// to sizes and offsets that the calls refuse, and stays small in ragged batches; lengths of any value stay within
// 31 bits.  Prints "ok" and exits 0.
#include <algorithm>
#include <climits>
#include <cstdio>
#include <memory>
#include <vector>

#include "attention_work.h"
#include "kv_internal.h"

static int failures = 0;
static void expect(const char *what, bool ok) {
    if (!ok && ++failures < 20) std::printf("FAIL %s\n", what);
}

static gdn_kv_args sizes() {
    gdn_kv_args a{};
    a.n_seqs = 2;
    a.n_heads = 8;
    a.n_kv_heads = 2;
    a.head_dim = 128;
    a.n_tokens = 5;
    a.n_pages = 4;
    a.page_tokens = 64;
    a.max_pages = 4096;
    a.n_layers = 1;
    a.in_dtype = GDN_BF16;
    return a;
}

static void check_refusals() {
    std::unique_ptr<int32_t[]> offs(new int32_t[3]{0, 3, 5});
    auto bytes = [&](auto edit) {
        gdn_kv_args a = sizes();
        edit(a);
        return gdn_attention_workspace_bytes(&a, offs.get());
    };
    expect("valid sizes need some", bytes([](gdn_kv_args &) {}) > 0);
    expect("head_dim", bytes([](gdn_kv_args &a) { a.head_dim = 96; }) == 0);
    expect("negative head_dim", bytes([](gdn_kv_args &a) { a.head_dim = -64; }) == 0);
    expect("dtype", bytes([](gdn_kv_args &a) { a.in_dtype = 2; }) == 0);
    expect("page_tokens", bytes([](gdn_kv_args &a) { a.page_tokens = 48; }) == 0);
    expect("n_pages", bytes([](gdn_kv_args &a) { a.n_pages = 0; }) == 0);
    expect("capacity", bytes([](gdn_kv_args &a) { a.max_pages = INT_MAX; }) == 0);
    expect("n_tokens", bytes([](gdn_kv_args &a) { a.n_tokens = 6; }) == 0);
    offs[2] = 1 << 30;
    expect("tokens beyond 30 bits", bytes([](gdn_kv_args &a) { a.n_tokens = 1 << 30, a.n_heads = a.n_kv_heads = 1; }) == 0);
    offs[2] = 5;
    expect("no tokens", bytes([](gdn_kv_args &a) { a.n_tokens = 0; }) == 0);
    expect("layers", bytes([](gdn_kv_args &a) { a.n_layers = 0; }) == 0);
    expect("layer_begin", bytes([](gdn_kv_args &a) { a.layer_begin = -1; }) == 0);
    expect("n_seqs", bytes([](gdn_kv_args &a) { a.n_seqs = INT_MAX; }) == 0);
    expect("no query heads", bytes([](gdn_kv_args &a) { a.n_heads = 0; }) == 0);
    expect("rows beyond 31 bits", bytes([](gdn_kv_args &a) { a.n_heads = 1 << 30; }) == 0);
    expect("too many layers", bytes([](gdn_kv_args &a) { a.n_layers = INT_MAX; }) == 0);
    expect("too many heads and layers", bytes([](gdn_kv_args &a) {
               a.n_heads = a.n_kv_heads = 400000000;
               a.n_layers = INT_MAX;
           }) == 0);
    offs[1] = 6;
    expect("decreasing offsets", bytes([](gdn_kv_args &) {}) == 0);
    offs[1] = -1;
    expect("negative offsets", bytes([](gdn_kv_args &) {}) == 0);
    offs[1] = offs[2] = 0;
    expect("offsets that hold no rows", bytes([](gdn_kv_args &) {}) == 0);
    expect("no rows at all", bytes([](gdn_kv_args &a) { a.n_tokens = 0; }) == 0);
}

// Batches whose rows are mostly one sequence's: the workspace holds what the device's workgroups can
// fill, a few fragments each, not a share of every unit that the longest sequence would have.
static void check_ragged() {
    for (int d : {64, 128, 256})
        for (int dtype : {GDN_F32, GDN_BF16})
            for (int heads : {1, 2, 8})
                for (int group : {1, 4, 8})
                    for (int seqs : {2, 8, 64, 300})
                        for (int longest : {2, 22, 100, 512, 3000})
                            for (int len : {1000, 3800, 20000, 200000}) {
                                gdn_kv_args a = sizes();
                                a.head_dim = d;
                                a.in_dtype = dtype;
                                a.n_seqs = seqs;
                                a.n_kv_heads = heads;
                                a.n_heads = heads * group;
                                a.n_tokens = seqs - 1 + longest;
                                a.max_length = len;
                                std::vector<int32_t> offs{0, longest};
                                while (int(offs.size()) <= seqs) offs.push_back(offs.back() + 1);
                                const gdn::AttentionPlan p = gdn::plan_attention(&a, offs.data());
                                const int64_t each = int64_t(2) * p.tile_rows * (d + 2) * 4;
                                expect("workgroups", p.parts <= 1 || p.workgroups <= 2 * 768);
                                expect("workspace", p.workspace <= 2 * 768 * each + p.units * 8);
                                expect("the query's size", int64_t(gdn_attention_workspace_bytes(&a, offs.data())) == p.workspace);
                            }
    // one of 800 new tokens and 99 of one
    gdn_kv_args a = sizes();
    a.n_seqs = 100;
    a.n_kv_heads = 1;
    a.n_tokens = 899;
    a.max_length = 3800;
    std::vector<int32_t> offs{0, 800};
    while (int(offs.size()) <= 100) offs.push_back(offs.back() + 1);
    expect("a prompt among single tokens", gdn_attention_workspace_bytes(&a, offs.data()) < (size_t(64) << 20));
}

// Lengths as they may lie on the device, up to the largest integers, with capacities up to 2^30.
static void check_lengths() {
    for (int64_t capacity : {int64_t(16), int64_t(4096), int64_t(1) << 30})
        for (int64_t length : {int64_t(INT_MIN), int64_t(-1), int64_t(0), int64_t(15), capacity - 1, capacity, int64_t(INT_MAX)}) {
            const int past = gdn::length_of(length, capacity);
            expect("length", past == std::max<int64_t>(0, std::min(length, capacity)));
            for (int node : {0, 1, 40, (1 << 30) - 2}) {
                expect("slots seen", gdn::slots_upto(past, node, capacity) == std::min(capacity, int64_t(past) + node + 1));
                expect("a node's slot in 31 bits", past + node + 1 > 0);
            }
        }
}

int main() {
    check_refusals();
    check_lengths();
    check_ragged();
    if (failures) return 1;
    std::printf("ok\n");
    return 0;
}
