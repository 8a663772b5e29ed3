"""Page tables and slot maps built on the device against the oracle: all values are equal."""
import numpy as np
import pytest

from gated_deltanet_tree_amd import binding
from oracle import kv as okv
from oracle import pages as op

import kv_harness as kh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    binding.lib()
    return torch


class Pool:
    """A pool whose sequences hold pages for `past` tokens, beside the oracle's lists."""

    def __init__(self, torch, past, new, page, n_pages, width, rng, share=0, depth=None):
        self.torch, self.page, self.past, self.new = torch, page, list(past), list(new)
        order = rng.permutation(n_pages).tolist()
        self.table, at = [], 0
        for p in past:
            n = min(width, -(-p // page))
            self.table.append(order[at:at + n] + [-1] * (width - n))
            at += n
        self.refs = [0] * n_pages
        for b in range(1, len(past)):  # some begin with the first one's pages
            for i in range(min(share, past[0] // page, past[b] // page)):
                self.table[b][i] = self.table[0][i]
        for row in self.table:
            for p in row:
                if p >= 0:
                    self.refs[p] += 1
        self.depth = depth
        self.pages, self.rc = kh.dev_i32(torch, self.table), kh.dev_i32(torch, self.refs)
        self.length = kh.dev_i32(torch, self.past)
        T, offs = sum(new), kh.offsets(new)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.missing, self.positions = torch.full((len(past),), -9, **i32), torch.full((T,), -9, **i32)
        self.slots = torch.full((T,), -9, dtype=torch.int64, device="cuda")
        kw = dict(missing=self.missing, slots=self.slots, positions=self.positions,
                  depth=None if depth is None else kh.dev_i32(torch, depth))
        a = (self.pages, self.length, self.rc, page, offs, kh.dev_i32(torch, offs))
        ws = torch.full((binding.pages_workspace_bytes(binding.pages_args(*a, **kw)),), 0xA5, dtype=torch.uint8,
                        device="cuda")
        self.args = binding.pages_args(*a, workspace=ws, **kw)

    def spoil(self, b, i, bad):
        """An entry that is no page's, its reference gone."""
        if 0 <= self.table[b][i] < len(self.refs):
            self.refs[self.table[b][i]] -= 1
        self.table[b][i] = bad
        self.pages.copy_(kh.dev_i32(self.torch, self.table))
        self.rc.copy_(kh.dev_i32(self.torch, self.refs))

    def same(self):
        self.torch.cuda.synchronize()
        assert self.pages.cpu().numpy().tolist() == self.table
        assert self.rc.cpu().numpy().tolist() == self.refs

    def reserve(self, stream=None):
        binding.kv_reserve(self.args, stream=stream)
        missing, slots, positions = op.reserve(self.table, self.refs, self.past, self.new, self.page, self.depth)
        self.same()
        assert self.missing.cpu().numpy().tolist() == missing
        assert self.slots.cpu().numpy().tolist() == slots
        assert self.positions.cpu().numpy().tolist() == positions
        return missing

    def release(self, keep, stream=None):
        binding.kv_release(self.args, kh.dev_i32(self.torch, keep), stream=stream)
        op.release(self.table, self.refs, keep, self.page)
        self.same()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("n_pages", [200, 2048, 2049, 9000])
def test_ragged_batches(torch, page, n_pages):
    rng = np.random.default_rng(page + n_pages)
    past = [0, 1, page - 1, page, page + 1, 5 * page, 7 * page + 3, 0]
    new = [0, 1, 1, 1, page, 3 * page + 1, 0, 2 * page]
    pool = Pool(torch, past, new, page, n_pages, 12, rng)
    assert not any(pool.reserve())
    pool.release([min(p + n, p + 2) for p, n in zip(past, new)])
    pool.reserve()
    pool.release([0] * 8)
    assert not any(pool.refs)


def test_free_pages_run_out(torch):
    rng = np.random.default_rng(0)
    pool = Pool(torch, [40, 0, 100, 7], [30, 100, 30, 300], 16, 20, 30, rng)
    missing = pool.reserve()
    assert missing[0] == 0 and sum(missing) > 0 and missing[3] > 0
    pool.release([0, 1000, 1000, 1000])  # one ends, and the others go on
    assert sum(pool.reserve()) > 0
    pool.release([0, 0, 0, 0])


@pytest.mark.parametrize("n_pages", [1, 20])
def test_no_free_page_at_all(torch, n_pages):
    rng = np.random.default_rng(1)
    pool = Pool(torch, [16 * n_pages], [1], 16, n_pages, 40, rng)
    assert pool.reserve() == [1]
    pool.release([16 * n_pages - 3])


def test_entries_that_hold_no_page_anywhere_are_filled(torch):
    """Holes in the middle of a table, ids out of range; what lies behind the need is left alone."""
    rng = np.random.default_rng(2)
    pool = Pool(torch, [100, 300, 50], [4, 1, 0], 16, 64, 25, rng)
    for b, i, bad in ((0, 0, -7), (0, 3, 64), (1, 5, 2**31 - 1), (1, 24, -5), (2, 1, -1), (2, 9, 10**6)):
        pool.spoil(b, i, bad)
    pool.reserve()
    pool.release([40, 0, 1000])


def test_shared_pages_are_free_when_nobody_holds_them(torch):
    rng = np.random.default_rng(3)
    pool = Pool(torch, [100, 200, 90, 64], [3, 3, 3, 3], 16, 80, 20, rng, share=4)
    assert max(pool.refs) == 4
    pool.reserve()
    pool.release([0, 203, 20, 0])
    pool.reserve()
    pool.release([0] * 4)
    assert not any(pool.refs)


def test_the_same_page_twice_and_references_that_were_lost(torch):
    """Counts do not go below zero."""
    rng = np.random.default_rng(4)
    pool = Pool(torch, [64, 32], [0, 0], 16, 9, 6, rng)
    pool.table[0][1] = pool.table[0][0]
    pool.pages.copy_(kh.dev_i32(torch, pool.table))
    pool.release([0, 0])


def test_lengths_below_zero_and_past_the_table(torch):
    rng = np.random.default_rng(5)
    pool = Pool(torch, [0, 0, 0], [20, 3, 3], 16, 300, 5, rng)
    pool.past = [-5, 75, 2**31 - 2]
    pool.length.copy_(kh.dev_i32(torch, pool.past))
    binding.kv_reserve(pool.args)
    missing, slots, positions = op.reserve(pool.table, pool.refs, pool.past, pool.new, 16)
    pool.same()
    assert pool.slots.cpu().numpy().tolist() == slots
    assert pool.positions.cpu().numpy().tolist() == [min(p, 2**31 - 1) for p in positions]
    pool.release([-3, 2**31 - 1, 80])


def test_depths_of_draft_trees(torch):
    rng = np.random.default_rng(6)
    trees = [kh.random_tree(rng, n) for n in (22, 1, 64)]
    image = binding.hld_schedule(trees)
    depth = binding.schedule_view(image)["node_depth"].tolist()
    pool = Pool(torch, [100, 15, 7], [22, 1, 64], 16, 100, 12, rng, depth=depth)
    pool.reserve()
    assert pool.positions.max().item() < 100 + 22


@pytest.mark.parametrize("S", [1, 63, 1024, 1025, 2500])
def test_many_sequences(torch, S):
    rng = np.random.default_rng(S)
    past, new = rng.integers(0, 70, S).tolist(), rng.integers(0, 40, S).tolist()
    pool = Pool(torch, past, new, 16, 8 * S + 5, 8, rng)
    pool.reserve()
    pool.release([p + n // 2 for p, n in zip(past, new)])
    pool.reserve()


def test_a_large_pool_and_long_tables(torch):
    rng = np.random.default_rng(7)
    pool = Pool(torch, [30000, 0, 12345], [4000, 9000, 1], 16, 300001, 2600, rng)
    pool.reserve()
    pool.release([100, 9000, 0])
    pool.reserve()


def test_outputs_may_be_left_out_and_other_streams(torch):
    rng = np.random.default_rng(8)
    pool = Pool(torch, [20, 5], [7, 30], 16, 30, 6, rng)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    pool.reserve(stream=s)
    pool.release([20, 5], stream=s)
    for n in ("missing", "slots", "positions"):
        setattr(pool.args, n, None)
    binding.kv_reserve(pool.args)
    op.reserve(pool.table, pool.refs, pool.past, pool.new, 16)
    pool.same()


def test_captured_steps_let_the_cache_grow(torch):
    """reserve, append, attend, commit and release in one graph: tables that begin empty fill as the
    lengths grow, and what the cache holds is what was appended."""
    S, H, d, page, width, n_new = 3, 2, 64, 16, 8, 4
    rng = np.random.default_rng(9)
    kv = binding.alloc_kv_cache(1, S, H, d, 20, page, width)
    refs = binding.alloc_kv_refs(kv)
    offs = np.arange(S + 1, dtype=np.int32) * n_new
    dev_offs = kh.dev_i32(torch, offs)
    f = dict(dtype=torch.bfloat16, device="cuda")
    k, v, q, out = (torch.zeros((1, S * n_new, h, d), **f) for h in (H, H, 4, 4))
    slots = torch.zeros(S * n_new, dtype=torch.int64, device="cuda")
    missing = torch.zeros(S, dtype=torch.int32, device="cuda")
    base = (kv.pages, kv.length, refs, page, offs, dev_offs)
    ws = torch.zeros(binding.pages_workspace_bytes(binding.pages_args(*base)), dtype=torch.uint8, device="cuda")
    ga = binding.pages_args(*base, missing=missing, slots=slots, workspace=ws)
    need = binding.attention_workspace_bytes(binding.kv_args(kv, offs, dev_offs, q=q, k=k, v=v, out=out))
    ka = binding.kv_args(kv, offs, dev_offs, q=q, k=k, v=v, out=out,
                         workspace=torch.zeros(need + 16, dtype=torch.uint8, device="cuda"))
    counts = torch.zeros(S, dtype=torch.int32, device="cuda")

    def step():
        binding.kv_reserve(ga)
        binding.kv_append(ka)
        binding.attention(ka)
        binding.kv_commit(ka, None, counts, kv.length)
        binding.kv_release(ga, kv.length)

    step()  # nothing is committed
    torch.cuda.synchronize()
    assert (kv.pages == -1).all() and not refs.any()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    hist = [[np.zeros((0, H, d))] * 2 for _ in range(S)]
    table, count, length = [[-1] * width for _ in range(S)], [0] * 20, [0] * S
    for i in range(30):
        ki, vi = (kh.rng_rows(rng, (S * n_new, H, d), "bf16") for _ in range(2))
        qi = kh.rng_rows(rng, (S * n_new, 4, d), "bf16", 1.5)
        take = rng.integers(0, n_new + 1, S)
        for t, y in ((k, ki), (v, vi), (q, qi)):
            t.copy_(kh.to_dev(torch, y[None], "bf16"))
        counts.copy_(kh.dev_i32(torch, take))
        graph.replay()
        torch.cuda.synchronize()
        short, want, _ = op.reserve(table, count, length, [n_new] * S, page)
        assert not any(short) and missing.cpu().numpy().tolist() == short
        assert slots.cpu().numpy().tolist() == want
        ks, vs = okv.stored_pair(ki, vi)
        got = kh.host(out[0])
        for b in range(S):
            sl = slice(b * n_new, (b + 1) * n_new)
            K, V = np.concatenate([hist[b][0], ks[sl]]), np.concatenate([hist[b][1], vs[sl]])
            kh.check_rows(qi[sl], got[sl], K, V, okv.visible_causal(length[b], n_new), d ** -0.5, "bf16")
            length[b] += int(take[b])
            hist[b] = [K[:length[b]], V[:length[b]]]
        op.release(table, count, length, page)
        assert kv.pages.cpu().numpy().tolist() == table and refs.cpu().numpy().tolist() == count
        assert kv.length.cpu().numpy().tolist() == length
        if max(length) > (width - 1) * page:
            break
    assert max(length) > 2 * page


@pytest.mark.parametrize("seqs,new,n_pages,width", [
    (96, 1, 8192, 170), (97, 1, 8192, 168), (64, 64, 8192, 256), (1, 1024, 8192, 16384), (1, 1025, 8192, 16384),
    (3, 341, 8192, 400), (3, 342, 8192, 400), (17, 64, 8193, 200), (16, 65, 4000, 1024), (96, 43, 3000, 100)])
def test_both_sides_of_what_one_launch_takes(torch, seqs, new, n_pages, width):
    """Sequences, tokens in all and on average, pages and entries up to its limits, and just beyond."""
    rng = np.random.default_rng(seqs + new)
    most = max(1, min(width, n_pages // seqs) * 16 - new - 40)
    past = rng.integers(0, most + 1, seqs).tolist()
    pool = Pool(torch, past, [new] * seqs, 16, n_pages, width, rng)
    pool.reserve()
    pool.release([p + 1 for p in past])
    pool.reserve()
    pool.release([0] * seqs)


def test_captured_reservations_of_many_sequences(torch):
    """The form in three launches, captured with its release, while lengths and tables change between replays."""
    rng = np.random.default_rng(8)
    S, page = 150, 16
    past = rng.integers(0, 200, S).tolist()
    new = rng.integers(0, 20, S).tolist()
    pool = Pool(torch, past, new, page, 4000, 40, rng)
    keep = torch.zeros(S, dtype=torch.int32, device="cuda")
    graph, give_back = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.kv_reserve(pool.args)
    with torch.cuda.graph(give_back):
        binding.kv_release(pool.args, keep)
    for step in range(12):
        pool.length.copy_(kh.dev_i32(torch, pool.past))
        graph.replay()
        missing, slots, positions = op.reserve(pool.table, pool.refs, pool.past, new, page)
        pool.same()
        assert pool.missing.cpu().numpy().tolist() == missing
        assert pool.slots.cpu().numpy().tolist() == slots and pool.positions.cpu().numpy().tolist() == positions
        pool.past = [0 if rng.random() < 0.1 else p + int(rng.integers(0, n + 1)) for p, n in zip(pool.past, new)]
        keep.copy_(kh.dev_i32(torch, pool.past))
        give_back.replay()
        op.release(pool.table, pool.refs, pool.past, page)
        pool.same()
