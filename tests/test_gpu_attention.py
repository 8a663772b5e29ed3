"""Attention over the 4-bit cache against the oracle, within the bound derived in kv_harness.py."""
import numpy as np
import pytest

from gated_deltanet_tree_amd import binding

import kv_harness as kh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    binding.lib()
    return torch


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 4, 6, 16])
def test_single_tokens(torch, d, dtype, group):
    """One new token a sequence, caches from none to several tiles, one sequence without any."""
    past = [0, 1, 15, 16, 31, 32, 33, 63, 64, 100, 257, 40]
    new = [1] * 11 + [0]
    c = kh.Cache(torch, past, new, kv_heads=2, d=d, dtype=dtype, seed=group, page=32)
    c.append_new()
    q, out = c.attend(2 * group)
    c.check(q, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 128])
def test_prompts(torch, d, dtype, page):
    """Ragged prompts from an empty and a filled cache, rows that end inside a tile."""
    past, new = [0, 0, 45, 7, 200], [1, 33, 70, 16, 29]
    c = kh.Cache(torch, past, new, kv_heads=2, d=d, dtype=dtype, seed=page, page=page, layers=2, layer=1)
    c.append_new()
    q, out = c.attend(6)
    c.check(q, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_trees(torch, d, dtype):
    """Trees of 1 to 130 nodes whose tails start anywhere in a tile."""
    rng = np.random.default_rng(d)
    sizes, past = [1, 2, 7, 22, 33, 64, 130], [3, 0, 31, 77, 64, 40, 21]
    trees = [kh.random_tree(rng, n, 4, 20) for n in sizes]
    c = kh.Cache(torch, past, sizes, kv_heads=2, d=d, dtype=dtype, seed=3)
    c.append_new()
    q, out = c.attend(6, trees=trees)
    c.check(q, out, trees=trees)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group,new", [(1, 7), (1, 8), (8, 1), (3, 3), (9, 1), (4, 4), (16, 1), (17, 1)])
def test_few_rows_of_32_bits(torch, d, group, new):
    """Row counts on both sides of a quarter and a half of a tile: ragged, whole and cut over
    workgroups, with a page that is not there, and as a tree."""
    past, news = [2500, 0, 61, 18], [new, new, max(new - 2, 0), 1]
    c = kh.Cache(torch, past, news, kv_heads=2, d=d, dtype="f32", page=32, seed=group, spare=0,
                 missing=[(0, 3, -1), (2, 1, -1)])
    c.append_new()
    q, out = c.attend(2 * group)
    c.check(q, out)
    q, out = c.attend(2 * group, max_length=40, q_scale=20.0)
    c.check(q, out)
    if 0 in news:  # a tree has a node
        return
    rng = np.random.default_rng(d)
    trees = [kh.random_tree(rng, n, 3, 5) for n in news]
    q, out = c.attend(2 * group, trees=trees)
    c.check(q, out, trees=trees)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group,new", [(1, 1), (4, 1), (3, 5), (16, 1), (2, 8)])
def test_few_rows_of_16_bits_keep_what_rounding_leaves_of_the_weights(torch, d, group, new):
    """Up to 16 rows: a weight enters as its rounding and the rounding of the rest, off by 2^-8 of
    2^-8 of it, flat and peaked scores, ragged, and cut over workgroups."""
    past, news = [2300, 0, 61, 18], [new, new, max(new - 1, 1), 1]
    c = kh.Cache(torch, past, news, kv_heads=2, d=d, dtype="bf16", page=32, seed=group)
    c.append_new()
    for q_scale in (1.0, 4.0):
        q, out = c.attend(2 * group, q_scale=q_scale)
        for b, o in enumerate(kh.offsets(news)[:-1]):
            kh.check_rows(q[o:o + news[b]], out[o:o + news[b]], c.K[b], c.V[b], c.visible(b), d ** -0.5, "bf16",
                          weight_half=2.0 ** -16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_token_that_is_not_finite_among_few_rows(torch, dtype):
    """The terms of a NaN score meet in its own row only."""
    tree = np.array([-1, 0, 0], dtype=np.int32)
    for group in (2, 5):
        c = kh.Cache(torch, [70], [3], kv_heads=2, d=64, dtype=dtype)
        k, v = c.rows(3), c.rows(3)
        k[1, 0, 5], v[2, 1, 7] = np.nan, np.inf
        c.append_new(k, v)
        q, out = c.attend(2 * group, trees=[tree])
        bad = np.zeros((3, 2 * group), dtype=bool)
        bad[1, :group] = bad[2, group:] = True
        assert np.isnan(out[bad]).all() and np.isfinite(out[~bad]).all()


def test_chain_and_star_trees_of_the_largest_size(torch):
    """A 1024-node chain (the causal call computes the same rows) and a 1024-node star."""
    chain, star = np.arange(-1, 1023, dtype=np.int32), np.array([-1] + [0] * 1023, dtype=np.int32)
    c = kh.Cache(torch, [10], [1024], kv_heads=1, d=64, page=64)
    c.append_new()
    q, out = c.attend(1, trees=[chain])
    _, causal = c.attend(1, q=q)
    c.check(q, out, trees=[chain])
    c.check(q, causal)
    q, out = c.attend(1, trees=[star])
    c.check(q, out, trees=[star])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 30])
def test_split_over_workgroups(torch, d, dtype, new):
    """Long caches of few rows are cut over workgroups and joined; any expected length gives
    results within the bound, and a call is repeatable bit for bit."""
    c = kh.Cache(torch, [3000, 17], [new, new], kv_heads=1, d=d, dtype=dtype, page=64)
    c.append_new()
    q = None
    for max_length in (0, 1, 300, 1500, 3030):
        q, out = c.attend(4, max_length=max_length, q=q)
        c.check(q, out)
        assert np.array_equal(out, c.attend(4, max_length=max_length, q=q)[1])


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64), ("f32", 128),
                                     ("f32", 256)])
def test_many_rows(torch, dtype, d):
    """Enough rows to fill the device without cutting the caches."""
    S = 70
    rng = np.random.default_rng(1)
    past, new = rng.integers(0, 50, S).tolist(), rng.integers(0, 45, S).tolist()
    c = kh.Cache(torch, past, new, kv_heads=8, d=d, dtype=dtype, page=16)
    c.append_new()
    q, out = c.attend(24)
    for b in (0, 1, 33, S - 1):  # every sequence is computed, a few are checked
        o = kh.offsets(new)[b]
        if new[b]:
            kh.check_rows(q[o:o + new[b]], out[o:o + new[b]], c.K[b], c.V[b], c.visible(b), d ** -0.5, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tree", [False, True])
def test_ragged_lengths_shared_out_as_one_line(torch, dtype, d, tree):
    """One long sequence among short and empty ones, enough units that every workgroup walks a share
    of all their tiles: shares begin and end inside units, and hold many units that have nothing."""
    S, group, rng = 62, 3, np.random.default_rng(d)
    past = [int(x) for x in rng.integers(0, 40, S)]
    past[40], past[0], past[61] = 2600, 0, 700
    new = [int(x) for x in rng.integers(1 if tree else 0, 5, S)]
    new[40], new[5], new[6] = 25 if dtype == "bf16" and d < 256 else 4, 1, 1
    c = kh.Cache(torch, past, new, kv_heads=8, d=d, dtype=dtype, page=128)
    c.append_new()
    trees = [kh.random_tree(rng, n, 3, 4) for n in new] if tree else None
    # more units than half the workgroups: cut they can only be as a line
    shape = kh.to_dev(torch, np.zeros((1, sum(new), 8 * group, d)), dtype)
    assert binding.attention_workspace_bytes(c.args(new, q=shape, out=shape)) > 0
    q, out = c.attend(8 * group, trees=trees)
    for b in (0, 5, 39, 40, 41, S - 1):
        o = kh.offsets(new)[b]
        if new[b]:
            kh.check_rows(q[o:o + new[b]], out[o:o + new[b]], c.K[b], c.V[b], c.visible(b, trees), d ** -0.5,
                          dtype)
    assert np.isfinite(out).all()
    assert np.array_equal(out, c.attend(8 * group, trees=trees, q=q)[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("max_length", [0, 30])
def test_rows_behind_the_last_sequence_are_left_alone(torch, dtype, max_length):
    """A batch padded to more rows than its offsets hold, whole and cut over workgroups."""
    past, new, pad = [2000, 3, 70], [1, 4, 12], 9
    c = kh.Cache(torch, past, new, kv_heads=2, d=128, dtype=dtype, page=64)
    c.append_new()
    T = sum(new)
    q = kh.rng_rows(c.rng, (T + pad, 8, 128), dtype, 1.5)
    qd = kh.to_dev(torch, q[None], dtype)
    out = torch.full_like(qd, 3.0)
    kw = dict(q=qd, out=out, max_length=max_length)
    need = binding.attention_workspace_bytes(c.args(new, **kw))
    ws = torch.empty((need // 4 + 4,), device="cuda")
    binding.attention(c.args(new, workspace=ws, **kw))
    torch.cuda.synchronize()
    assert (out[0, T:] == 3.0).all()
    c.check(q[:T], kh.host(out[0, :T]))


def test_wide_and_flat_scores(torch):
    """Score ranges from nearly equal to a single winner, and a winner at every position."""
    for q_scale in (1e-3, 1.0, 30.0):
        c = kh.Cache(torch, [150], [3], kv_heads=1, d=128, dtype="f32", seed=5)
        c.append_new()
        q, out = c.attend(4, q_scale=q_scale)
        c.check(q, out)
    c = kh.Cache(torch, [0], [96], kv_heads=1, d=64, dtype="bf16")
    k = np.zeros((96, 1, 64))
    k[np.arange(96), 0, np.arange(96) % 64] = 6.0
    c.append_new(k, None)
    q = np.zeros((96, 1, 64))
    q[np.arange(96), 0, (np.arange(96) * 7) % 64] = 40.0
    _, out = c.attend(1, q=q)
    c.check(q, out)


def test_missing_pages_leave_rows_empty(torch):
    """Pages that are not there are not seen; a row that sees nothing is zero."""
    past, new = [0, 40, 100, 64], [5, 20, 3, 4]
    c = kh.Cache(torch, past, new, kv_heads=2, d=128, dtype="f32", spare=0,
                 missing=[(0, 0, -1), (1, 1, 1 << 29), (2, 0, -1), (2, 6, -1)] +
                         [(3, i, -1) for i in range(5)])
    c.append_new()
    q, out = c.attend(4)
    c.check(q, out)
    assert (out[:5] == 0).all() and (out[-4:] == 0).all()


def test_poisoned_tokens_reach_only_rows_that_see_them(torch):
    """A NaN in one branch of a tree, an infinity in another: their rows and their descendants' are
    NaN, siblings and other heads are untouched."""
    tree = np.array([-1, 0, 0, 1, 2, 3, 4, 4], dtype=np.int32)
    c = kh.Cache(torch, [37], [8], kv_heads=2, d=128, dtype="bf16")
    k, v = c.rows(8), c.rows(8)
    k[1, 0, 5], v[4, 1, 100] = np.nan, np.inf
    c.append_new(k, v)
    q, out = c.attend(6, trees=[tree])
    c.check(q, out, trees=[tree])
    bad = np.isnan(out).any(-1)
    assert sorted(set(np.flatnonzero(bad[:, 0]))) == [1, 3, 5]
    assert sorted(set(np.flatnonzero(bad[:, 5]))) == [4, 6, 7]


def test_lengths_out_of_range(torch):
    """A negative length counts as 0; one at the capacity sees the table and drops the new rows."""
    c = kh.Cache(torch, [0, 32], [4, 2], kv_heads=1, d=64, dtype="f32", spare=0)
    c.append_new()
    c.kv.length.copy_(torch.tensor([-9, 32], dtype=torch.int32))
    q, out = c.attend(2)
    c.check(q, out)
    full = c.table.shape[1] * 16
    c2 = kh.Cache(torch, [full], [0], kv_heads=1, d=64, dtype="f32", spare=0)
    c2.new, c2.past = [3], [full]
    c2.table = c2.table[:, :full // 16]
    c2.kv.pages = c2.kv.pages[:, :full // 16].contiguous()
    c2.append([3], c2.rows(3), c2.rows(3))
    q, out = c2.attend(2)
    see = np.ones((3, full), dtype=bool)
    kh.check_rows(q, out, c2.K[0], c2.V[0], see, 64 ** -0.5, "f32")


def test_offsets_beyond_32_bits(torch):
    """A pool whose last pages lie past 4 GiB of codes: pages there are appended and read."""
    d, page, H = 256, 256, 8
    per_page = H * page * d // 2
    n_pages = (1 << 32) // per_page + 40
    kv = binding.alloc_kv_cache(1, 1, H, d, n_pages, page, 4)
    kv.pages.copy_(torch.tensor([[n_pages - 1, n_pages - 3, 0, n_pages - 2]], dtype=torch.int32))
    rng = np.random.default_rng(2)
    n = 700
    k, v = (kh.rng_rows(rng, (n, H, d), "bf16") for _ in range(2))
    offs = np.array([0, n], dtype=np.int32)
    kd, vd = kh.to_dev(torch, k[None], "bf16"), kh.to_dev(torch, v[None], "bf16")
    binding.kv_append(binding.kv_args(kv, offs, kh.dev_i32(torch, offs), k=kd, v=vd))
    q = kh.rng_rows(rng, (n, H, d), "bf16")
    out = torch.empty((1, n, H, d), dtype=torch.bfloat16, device="cuda")
    kw = dict(q=kh.to_dev(torch, q[None], "bf16"), out=out)
    need = binding.attention_workspace_bytes(binding.kv_args(kv, offs, kh.dev_i32(torch, offs), **kw))
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
    binding.attention(binding.kv_args(kv, offs, kh.dev_i32(torch, offs), workspace=ws, **kw))
    from oracle import kv as okv
    at = [0, 255, 256, 511, 512, 699]
    ks, vs = okv.stored_pair(k, v)
    see = okv.visible_causal(0, n)[at]
    kh.check_rows(q[at], kh.host(out[0])[at], ks, vs, see, d ** -0.5, "bf16")


def test_streams_and_graph_replay(torch):
    """On a side stream; captured and replayed with new rows, lengths and pages, with eager calls
    in between; two graphs with workspaces of their own."""
    past, new = [900, 12], [5, 5]
    c = kh.Cache(torch, past, new, kv_heads=1, d=128, dtype="bf16", page=64)
    c.append_new()
    q, eager = c.attend(4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert np.array_equal(c.attend(4, q=q, stream=s)[1], eager)
    graphs = []
    for _ in range(2):
        qd = kh.to_dev(torch, q[None], "bf16")
        out = torch.zeros_like(qd)
        need = binding.attention_workspace_bytes(c.args(new, q=qd, out=out))
        assert need > 0
        a = c.args(new, q=qd, out=out, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            binding.attention(a)
        graphs.append((g, qd, out, a))
    for step in range(3):
        c.append_new()
        q = kh.rng_rows(c.rng, q.shape, "bf16")
        for g, qd, out, _ in graphs:
            qd.copy_(kh.to_dev(torch, q[None], "bf16"))
            g.replay()
        torch.cuda.synchronize()
        _, eager = c.attend(4, q=q)
        c.check(q, eager)
        for _, _, out, _ in graphs:
            assert np.array_equal(kh.host(out[0]), eager)


def test_largest_group_and_odd_heads(torch):
    c = kh.Cache(torch, [50, 9], [3, 1], kv_heads=3, d=64, dtype="bf16")
    c.append_new()
    q, out = c.attend(3 * 37)  # rows of one token fill more than a tile
    c.check(q, out)


def _wide_table(torch, c, width):
    """The cache's sequences in a table of `width` entries, whose others are not there."""
    table = np.full((c.table.shape[0], width), -1, dtype=np.int32)
    table[:, :c.table.shape[1]] = c.table
    c.table = table
    c.kv.pages = torch.from_numpy(table).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 2])
def test_short_sequences_in_a_long_table(torch, d, dtype, group):
    """One kv head and a capacity of 262144 slots: a call of hundreds of parts, more than a short
    sequence costs, over a workspace of NaN."""
    for past in (0, 10, 50, 200, 470):
        c = kh.Cache(torch, [past], [1], kv_heads=1, d=d, dtype=dtype, page=64, seed=past)
        _wide_table(torch, c, 4096)
        c.append_new()
        q, out = c.attend(group)
        c.check(q, out)
        assert np.array_equal(out, c.attend(group, q=q)[1])
        _, out = c.attend(group, trees=[np.array([-1], dtype=np.int32)], q=q)
        c.check(q, out)


def test_a_short_sequence_beside_a_longer_one(torch):
    """The parts go by the longest sequence expected, of which one may have no new token."""
    for past, new in (([11, 2500], [1, 1]), ([7, 3000, 0], [1, 0, 1])):
        c = kh.Cache(torch, past, new, kv_heads=1, d=64, page=64)
        _wide_table(torch, c, 4096)
        c.append_new()
        q, out = c.attend(1, max_length=100001)
        c.check(q, out)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 128), ("f32", 256)])
def test_a_prompt_among_single_tokens(torch, dtype, d):
    """Most of the rows are one sequence's: whatever the length that is expected, the workspace stays
    within what the device's workgroups fill, and every row is right."""
    past, new = [70, 0, 33, 500, 12, 7, 64, 100, 31, 1], [1, 1, 100, 1, 1, 0, 1, 1, 1, 1]
    c = kh.Cache(torch, past, new, kv_heads=1, d=d, dtype=dtype, page=64)
    _wide_table(torch, c, 1024)
    c.append_new()
    q = None
    shape = kh.to_dev(torch, np.zeros((1, sum(new), 8, d)), dtype)
    for max_length in (0, 600, 3000, 12000):
        need = binding.attention_workspace_bytes(c.args(new, q=shape, out=shape, max_length=max_length))
        assert need <= 2 * 768 * 2 * 64 * (d + 2) * 4 + 8 * 10 * 100
        q, out = c.attend(8, max_length=max_length, q=q)
        c.check(q, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lengths_far_beyond_the_table(torch, dtype):
    """A length past the capacity, up to the largest integer, is the capacity: every row sees the whole
    table, of new tokens that have no slots."""
    c = kh.Cache(torch, [128, 48, 128], [1, 1, 1], kv_heads=2, d=64, dtype=dtype, page=16, spare=0)
    new = [3, 40, 1]
    c.new = new
    c.table = c.table[:, :8].copy()
    c.table[1, 3:] = -1
    c.kv.pages = torch.from_numpy(c.table).cuda()
    trees = [kh.random_tree(np.random.default_rng(1), n, 3, 9) for n in new]
    at = kh.offsets(new)
    for length in ([128, 131, 128], [129, 1 << 30, 4000], [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 31 - 40]):
        c.kv.length.copy_(torch.tensor(length, dtype=torch.int32))
        for group, tree in ((1, None), (9, None), (1, trees), (9, trees)):
            q, out = c.attend(2 * group, trees=tree)
            for b, n in enumerate(new):
                L = 128 if b != 1 else 48
                kh.check_rows(q[at[b]:at[b] + n], out[at[b]:at[b] + n], c.K[b][:L], c.V[b][:L],
                              np.ones((n, L), dtype=bool), 64 ** -0.5, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("group,new", [(1, 3), (6, 12)])
def test_infinities_and_nan_in_q_make_their_rows_nan(torch, dtype, d, group, new):
    """A score is then infinite or NaN, of either sign, and so no weight is a number; a row that sees
    nothing stays zero, and the other rows are right."""
    past = [0, 40, 5]
    c = kh.Cache(torch, past, [new] * 3, kv_heads=2, d=d, dtype=dtype, page=16, spare=0,
                 missing=[(2, i, -1) for i in range(-(-(5 + new) // 16))])
    c.append_new()
    q = kh.rng_rows(c.rng, (3 * new, 2 * group, d), dtype)
    bad = np.zeros(q.shape[:2], dtype=bool)
    for i, (row, head) in enumerate([(0, 0), (0, 2 * group - 1), (1, 0), (new - 1, group), (new, 0), (new + 1, group),
                                     (2 * new - 1, 1), (2 * new, 0), (3 * new - 1, group)]):
        q[row, head, (7 * i) % d] = (np.inf, -np.inf, np.nan)[i % 3]
        bad[row, head] = True
    # one channel of the only key a row sees, of either sign, decides the score's
    for chan in range(4):
        q[0, 0, :] = 0.25
        q[0, 0, chan] = -np.inf
        _, out = c.attend(2 * group, q=q)
        assert np.isnan(out[:2 * new][bad[:2 * new]]).all()
        assert (out[2 * new:] == 0).all()
        assert np.isfinite(out[:2 * new][~bad[:2 * new]]).all()
    good = np.where(bad[..., None], 0.0, q)
    _, want = c.attend(2 * group, q=good)
    assert np.array_equal(out[~bad], want[~bad])


@pytest.mark.parametrize("dtype,d,group", [("bf16", 64, 3), ("bf16", 128, 6), ("bf16", 256, 2), ("f32", 64, 9), ("f32", 128, 2)])
@pytest.mark.parametrize("max_length,past", [(100, [0, 37, 60]), (0, [3, 900, 20]), (60000, [30, 2, 1500])])
def test_several_layers_in_one_call(torch, dtype, d, group, max_length, past):
    """Layers 1 to 3 of 4: whole units, parts and shares of a line that runs through the layers; causal
    and trees; layer 0's output is left alone."""
    rng = np.random.default_rng(d + group)
    layers, heads, new = 4, 2, [2, 7, 4]
    S, T, L0 = 3, sum(new), max(p + n for p, n in zip(past, new))
    width = -(-L0 // 32) if max_length < 1000 else 2048
    used = -(-L0 // 32)
    kv = binding.alloc_kv_cache(layers, S, heads, d, S * used, 32, width)
    table = np.full((S, width), -1, dtype=np.int32)
    table[:, :used] = rng.permutation(S * used).reshape(S, used)
    kv.pages.copy_(torch.from_numpy(table))
    K, V = [[None] * S for _ in range(layers)], [[None] * S for _ in range(layers)]
    full = [p + n for p, n in zip(past, new)]
    at, offs = kh.offsets(full), kh.offsets(new)
    k, v = (kh.rng_rows(rng, (layers, sum(full), heads, d), dtype) for _ in range(2))
    binding.kv_append(binding.kv_args(kv, at, kh.dev_i32(torch, at), k=kh.to_dev(torch, k, dtype),
                                      v=kh.to_dev(torch, v, dtype), layer_begin=1, n_layers=3))
    from oracle import kv as okv
    kv.length.copy_(torch.tensor(past, dtype=torch.int32))
    trees = [kh.random_tree(rng, n, 3, 4) for n in new]
    image = binding.hld_schedule(trees)
    q = kh.rng_rows(rng, (layers, T, heads * group, d), dtype, 1.5)
    for tree in (False, True):
        qd = kh.to_dev(torch, q, dtype)
        out = torch.full_like(qd, 5.0)
        kw = dict(q=qd, out=out, max_length=max_length, layer_begin=1, n_layers=3)
        dev = kh.dev_i32(torch, offs)
        need = binding.attention_workspace_bytes(binding.kv_args(kv, offs, dev, **kw))
        ws = torch.full((need // 4 + 4,), float("nan"), device="cuda")
        a = binding.kv_args(kv, offs, dev, workspace=ws, **kw)
        if tree:
            binding.tree_attention(a, image, torch.from_numpy(image).cuda())
        else:
            binding.attention(a)
        torch.cuda.synchronize()
        got = kh.host(out)
        assert (got[0] == 5.0).all()
        for layer in (1, 2, 3):
            for b in range(S):
                if K[layer][b] is None:
                    K[layer][b], V[layer][b] = okv.stored_pair(k[layer, at[b]:at[b + 1]], v[layer, at[b]:at[b + 1]])
                see = okv.visible_tree(trees[b], past[b]) if tree else okv.visible_causal(past[b], new[b])
                rows = slice(offs[b], offs[b + 1])
                kh.check_rows(q[layer, rows], got[layer, rows], K[layer][b], V[layer][b], see, d ** -0.5, dtype)


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "f32")])
def test_captured_decode_while_a_cache_grows(torch, d, dtype):
    """One graph over a table of 262144 slots, replayed from an empty cache to one that costs more than
    the call has parts, with eager calls in between."""
    c = kh.Cache(torch, [1100], [1], kv_heads=1, d=d, dtype=dtype, page=64)
    _wide_table(torch, c, 4096)
    c.append_new()
    K, V = c.K[0], c.V[0]
    q = kh.rng_rows(c.rng, (1, 2, d), dtype, 1.5)
    qd = kh.to_dev(torch, q[None], dtype)
    out = torch.zeros_like(qd)
    need = binding.attention_workspace_bytes(c.args([1], q=qd, out=out))
    a = c.args([1], q=qd, out=out, workspace=torch.full((need // 4 + 4,), float("nan"), device="cuda"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.attention(a)
    for past in (0, 1, 30, 250, 251, 480, 1100, 3, 0):
        c.kv.length.fill_(past)
        g.replay()
        torch.cuda.synchronize()
        got = kh.host(out[0])
        kh.check_rows(q, got, K[:past + 1], V[:past + 1], np.ones((1, past + 1), dtype=bool), d ** -0.5, dtype)
        assert np.array_equal(got, c.attend(2, q=q)[1])
