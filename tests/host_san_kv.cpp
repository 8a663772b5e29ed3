// Driver of the 4-bit cache's address arithmetic and argument checks for the sanitized host build:
// every byte of a slab belongs to exactly one (token, channel group) or scale, pages that are not
// there and slots past the table are turned away before the table is read, and malformed arguments
// are refused without reading past the offsets.  Prints "ok" and exits 0.
#include <climits>
#include <cstdio>
#include <cstring>
#include <memory>
#include <vector>

#include "attention_work.h"
#include "kv_internal.h"
#include "kv_layout.h"

static int failures = 0;
static void expect(const char *what, bool ok) {
    if (!ok) {
        std::printf("FAIL %s (%s)\n", what, gdn_last_error());
        ++failures;
    }
}

// Counts how often each byte of a slab is addressed, in heap blocks of exactly the slab's size.
template <int D> static void check_layout(int page) {
    typedef gdn::KvAt<D> At;
    std::vector<int> kc(size_t(page) * D / 2), ks(size_t(page) * D / 32), vc(kc.size()), vs(ks.size());
    for (int t = 0; t < page; ++t) {
        for (int c = 0; c < D / 8; ++c)
            for (int x = 0; x < 4; ++x) ++kc.at(size_t(At::key(t, c) + x));
        for (int m = 0; m < 32; ++m)
            for (int x = 0; x < D / 64; ++x) ++vc.at(size_t(At::value(t, m) + x));
        for (int b = 0; b < D / 32; ++b) {
            ++ks.at(size_t(At::key_scale(t, b)));
            ++vs.at(size_t(At::value_scale(t, b)));
        }
        if (t % 4 == 0) {  // a quad's value pieces and scales are contiguous
            for (int i = 1; i < 4; ++i) {
                expect("value piece", At::value(t + i, 5) == At::value(t, 5) + i * (D / 64));
                expect("scale piece", At::value_scale(t + i, 1) == At::value_scale(t, 1) + i);
            }
        }
    }
    for (const auto *v : {&kc, &ks, &vc, &vs})
        for (int n : *v) expect("each byte once", n == 1);
}

static void check_pages() {
    std::unique_ptr<int32_t[]> table(new int32_t[5]{3, -1, 7, INT_MIN, INT_MAX});
    auto page = [&](int64_t pos) { return gdn::kv_page(table.get(), 5, 7, 4, pos); };
    expect("page in the pool", page(0) == 3 && page(15) == 3);
    expect("absent pages", page(16) == -1 && page(32) == -1 && page(48) == -1 && page(64) == -1);
    expect("past the table", page(80) == -1 && page(INT64_MAX) == -1 && page(-1) == -1);
    expect("large pools", gdn::kv_slab(40, 1 << 20, (1 << 20) - 1, 8, 7) == (41ll << 23) - 1);
}

static void check_exponents() {
    uint32_t bits;
    const struct { float amax; int e; } cases[] = {{0.f, -125}, {4.f, 0}, {7.f, 0}, {7.0001f, 1}, {3.4e38f, 125},
                                                   {1e-45f, -125}, {1.f, -2}};
    for (const auto &c : cases) {
        std::memcpy(&bits, &c.amax, 4);
        expect("scale exponent", gdn::kv_scale_exp(bits) == c.e);
    }
}

static gdn_kv_args valid() {
    gdn_kv_args a{};
    a.n_seqs = 2;
    a.n_heads = 8;
    a.n_kv_heads = 2;
    a.head_dim = 128;
    a.n_tokens = 5;
    a.n_pages = 4;
    a.page_tokens = 64;
    a.max_pages = 4;
    a.n_layers = 1;
    a.in_dtype = GDN_BF16;
    uint8_t *p = reinterpret_cast<uint8_t *>(4096);
    a.k_codes = a.v_codes = a.k_scales = a.v_scales = p;
    a.pages = a.length = a.seq_offsets = reinterpret_cast<int32_t *>(p);
    return a;
}

static void check_args() {
    std::unique_ptr<int32_t[]> offs(new int32_t[3]{0, 3, 5});
    bool empty;
    auto status = [&](const gdn_kv_args &a) { return gdn::check_kv_args(&a, offs.get(), "call", true, empty); };
    expect("valid", status(valid()) == GDN_OK && !empty);
    auto bad = [&](const char *what, auto edit) {
        gdn_kv_args a = valid();
        edit(a);
        expect(what, status(a) == GDN_EINVAL);
    };
    bad("head_dim", [](gdn_kv_args &a) { a.head_dim = 96; });
    bad("page_tokens", [](gdn_kv_args &a) { a.page_tokens = 48; });
    bad("page_tokens 0", [](gdn_kv_args &a) { a.page_tokens = 0; });
    bad("n_seqs", [](gdn_kv_args &a) { a.n_seqs = -1; });
    bad("n_seqs large", [](gdn_kv_args &a) { a.n_seqs = INT_MAX; });
    bad("n_pages", [](gdn_kv_args &a) { a.n_pages = 0; });
    bad("max_pages", [](gdn_kv_args &a) { a.max_pages = 0; });
    bad("capacity", [](gdn_kv_args &a) { a.max_pages = INT_MAX; });
    bad("n_kv_heads", [](gdn_kv_args &a) { a.n_kv_heads = 0; });
    bad("layers", [](gdn_kv_args &a) { a.n_layers = 0; });
    bad("layer_begin", [](gdn_kv_args &a) { a.layer_begin = -1; });
    bad("dtype", [](gdn_kv_args &a) { a.in_dtype = 2; });
    bad("n_tokens", [](gdn_kv_args &a) { a.n_tokens = 6; });
    bad("null pool", [](gdn_kv_args &a) { a.v_scales = nullptr; });
    bad("misaligned pool", [](gdn_kv_args &a) { a.k_codes += 8; });
    bad("null pages", [](gdn_kv_args &a) { a.pages = nullptr; });
    bad("null length", [](gdn_kv_args &a) { a.length = nullptr; });
    bad("null offsets", [](gdn_kv_args &a) { a.seq_offsets = nullptr; });
    offs[1] = 6;
    bad("decreasing offsets", [](gdn_kv_args &) {});
    offs[1] = 3;
    expect("null arguments", gdn::check_kv_args(nullptr, offs.get(), "call", true, empty) == GDN_EINVAL);
    const gdn_kv_args v = valid();
    expect("null host offsets", gdn::check_kv_args(&v, nullptr, "call", true, empty) == GDN_EINVAL);
}

// The work line: blocks partition a sequence's cost, positions find their block, shares cut every
// unit into runs of tiles that follow on one another.
static void check_work() {
    for (int64_t past : {0, 1, 31, 4000, 1 << 29})
        for (int64_t n : {0, 1, 22, 1000, 40000})
            for (int64_t group : {1, 6, 37})
                for (int64_t rows : {32, 64})
                    for (bool tree : {false, true}) {
                        const gdn::SeqWork s = gdn::seq_work(past, n, group, rows, tree, 1 << 30);
                        expect("blocks", s.blocks == (n * group + rows - 1) / rows);
                        expect("cost", s.cost == gdn::cost_before(s, s.blocks) && (s.cost > 0) == (n > 0));
                        for (int64_t k : {int64_t(0), int64_t(1), s.blocks / 2, s.blocks - 1}) {
                            if (k < 0 || k >= s.blocks) continue;
                            const int64_t at = gdn::cost_before(s, k), v = s.a + s.b * k;
                            expect("unit", at + v == gdn::cost_before(s, k + 1) && v > 0);
                            expect("first", gdn::block_at(s, at) == k);
                            expect("last", gdn::block_at(s, at + v - 1) == k);
                            for (int tiles : {0, 1, 7, 1 << 25}) {
                                int before = 0;
                                for (int i = 0; i <= 5; ++i) {
                                    const int t = gdn::tile_at(v * i / 5, v, tiles);
                                    expect("tiles in order", t >= before && t <= tiles);
                                    before = t;
                                }
                                expect("tiles end", before == tiles && gdn::tile_at(0, v, tiles) == 0);
                            }
                        }
                    }
    for (int64_t a : {int64_t(0), int64_t(1), int64_t(999), (int64_t(1) << 53) + 1, (int64_t(1) << 58) - 1})
        for (int64_t b : {int64_t(1), int64_t(2), int64_t(998), int64_t(1000), (int64_t(1) << 30) + 7})
            expect("quotient", gdn::quotient(a, b) == a / b);
    const gdn::SeqWork held = gdn::seq_work(100, 50, 2, 32, true, 64);  // lengths beyond the capacity
    expect("capacity", held.a == (64 + gdn::kUnitSlots) * 2 && gdn::seq_work(-5, 1, 1, 32, true, 64).a == 1 + gdn::kUnitSlots);
}

// Every plan covers the rows, stays within the launch limits and needs workspace only for shares.
static void check_plans() {
    for (int d : {64, 128, 256})
        for (int dtype : {GDN_F32, GDN_BF16})
            for (int seqs : {1, 3, 64})
                for (int n : {1, 7, 64, 3000})
                    for (int group : {1, 6, 40})
                        for (int len : {0, 1, 100, 100000}) {
                            gdn_kv_args a = valid();
                            a.head_dim = d;
                            a.in_dtype = dtype;
                            a.n_seqs = seqs;
                            a.n_tokens = seqs * n;
                            a.n_heads = 2 * group;
                            a.max_length = len;
                            a.max_pages = 4096;
                            std::vector<int32_t> offs;
                            for (int b = 0; b <= seqs; ++b) offs.push_back(b * n);
                            const gdn::AttentionPlan p = gdn::plan_attention(&a, offs.data());
                            const int64_t rows = int64_t(n) * group;
                            expect("rows covered", int64_t(p.row_blocks) * p.tile_rows >= rows &&
                                                       int64_t(p.row_blocks - 1) * p.tile_rows < rows);
                            expect("rows of a block", p.max_rows == (rows < p.tile_rows ? rows : p.tile_rows));
                            expect("workgroups", p.workgroups >= 1 && p.parts >= 0 &&
                                                     (p.parts == 0 || p.workgroups == p.units * p.parts) && p.units == int64_t(p.row_blocks) * seqs * 2);
                            expect("workspace", p.workspace == (p.parts == 1 ? 0 : p.units * 8 + p.workgroups * 2 * p.tile_rows * (d + 2) * 4) &&
                                                    int64_t(gdn_attention_workspace_bytes(&a, offs.data())) == p.workspace);
                        }
    gdn_kv_args a = valid();
    const int32_t offs[] = {0, 3, 5};
    a.n_heads = 7;
    expect("no plan for uneven heads", gdn_attention_workspace_bytes(&a, offs) == 0);
    expect("no plan for nothing", gdn_attention_workspace_bytes(nullptr, offs) == 0);
}

int main() {
    for (int page : {16, 32, 64, 128, 256}) {
        check_layout<64>(page);
        check_layout<128>(page);
        check_layout<256>(page);
    }
    check_pages();
    check_exponents();
    check_args();
    check_work();
    check_plans();
    if (failures) return 1;
    std::printf("ok\n");
    return 0;
}
