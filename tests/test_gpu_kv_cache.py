"""The 4-bit cache's append, commit and read against the oracle: stored values are equal, slots
nothing was written to keep their bytes."""
import numpy as np
import pytest

from gated_deltanet_tree_amd import binding, synth
from oracle import kv as okv

import kv_harness as kh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    binding.lib()
    return torch


def _read(c, counts, begin=None):
    T, torch = sum(counts), c.torch
    dt = torch.bfloat16 if c.dtype == "bf16" else torch.float32
    k = torch.full((c.layers, T, c.H, c.d), 7.0, device="cuda", dtype=dt)
    v = torch.full_like(k, 7.0)
    binding.kv_read(c.args(counts, k=k, v=v), begin=begin)
    torch.cuda.synchronize()
    for other in range(c.layers):
        if other != c.layer:
            assert (k[other] == 7.0).all() and (v[other] == 7.0).all()
    return kh.host(k[c.layer]), kh.host(v[c.layer])


def _pools(c):
    return [t.cpu().numpy().copy() for t in (c.kv.k_codes, c.kv.k_scales, c.kv.v_codes, c.kv.v_scales)]


def _written(c, before, slots):
    """Bytes outside the listed (sequence, slot) pairs of the layer in use are as before."""
    after = _pools(c)
    mask = [np.zeros(a.shape, dtype=bool) for a in after]
    for b, p in slots:
        pg = c.table[b, p // c.page]
        for m, at in zip(mask, kh.token_bytes(c.d, p % c.page)):
            m[c.layer, pg][:, at] = True
    for a, x, m in zip(after, before, mask):
        assert np.array_equal(a[~m], x[~m])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_append_and_read(torch, d, dtype, page):
    """Ragged starts and lengths: 0, 1, within and across quads, groups and pages."""
    past = [0, 1, 3, 15, 16, 17, 63, 100]
    new = [1, 2, 5, 1, 0, 33, 130, 4]
    c = kh.Cache(torch, past, new, kv_heads=3, d=d, page=page, dtype=dtype, seed=d + page, layers=2, layer=1)
    before = _pools(c)
    c.append_new()
    _written(c, before, [(b, p) for b in range(8) for p in range(past[b], past[b] + new[b])])
    k, v = _read(c, new)
    for b, o in enumerate(kh.offsets(new)[:-1]):
        assert np.array_equal(k[o:o + new[b]], c.K[b][past[b]:])
        assert np.array_equal(v[o:o + new[b]], c.V[b][past[b]:])
    # the whole sequences, from slot 0
    total = [p + n for p, n in zip(past, new)]
    k, v = _read(c, total, begin=torch.zeros(8, dtype=torch.int32, device="cuda"))
    assert np.array_equal(k, np.concatenate(c.K)) and np.array_equal(v, np.concatenate(c.V))


def test_every_bf16_value_rounds_to_the_nearest_code(torch):
    """Every finite bf16 value beside a block maximum of its own binade, the next and four above."""
    bits = np.arange(1 << 16, dtype=np.uint16)
    x = synth.bf16_to_f32(bits)
    x = x[np.isfinite(x)].astype(np.float64)
    rows = []
    for up in (0, 1, 4):
        blocks = np.zeros((len(x) // 31 + 1, 32))
        blocks[:, 1:].reshape(-1)[:] = 0
        flat = np.zeros(blocks.shape[0] * 31)
        order = np.argsort(np.abs(x), kind="stable")
        flat[:len(x)] = x[order]
        blocks[:, 1:] = flat.reshape(-1, 31)
        top = np.abs(blocks[:, 1:]).max(1)
        blocks[:, 0] = np.minimum(top * 2.0 ** up, 3.0e38)
        rows.append(blocks)
    x = np.concatenate(rows)
    x = synth.bf16_to_f32(synth.f32_to_bf16(np.minimum(x, 3.38e38).astype(np.float32))).astype(np.float64)
    x = np.concatenate([x, np.zeros((-len(x) % 4, 32))]).reshape(-1, 1, 128)
    for dtype in ("bf16", "f32"):
        c = kh.Cache(torch, [0], [len(x)], kv_heads=1, d=128, page=64, dtype=dtype)
        c.append_new(x, -x)
        k, v = _read(c, [len(x)])
        assert np.array_equal(k, c.K[0]) and np.array_equal(v, c.V[0])


def test_fp32_ties_and_their_neighbours(torch):
    """Midpoints of the grid and the fp32 values next to them, at many scales."""
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0], dtype=np.float32)
    vals = np.concatenate([mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(9))])
    rows = []
    for e in list(range(-126, 124, 7)) + [-126, 124]:
        with np.errstate(over="ignore"):
            r = np.zeros((1, 32), dtype=np.float64)
            r[0, :27] = vals.astype(np.float64) * 2.0 ** e
            r[0, 27:] = [4.0 * 2.0 ** e, -2.5 * 2.0 ** e, 0.0, -0.0, 1e-45]
        for top in (4.0, 6.0, 7.0, 7.000001):
            q = r.copy()
            q[np.abs(q) > top * 2.0 ** e] = 0.0
            q[0, 27] = top * 2.0 ** e
            rows.append(q.astype(np.float32).astype(np.float64))
    x = np.concatenate(rows)
    x = np.concatenate([x, np.zeros((-len(x) % 2, 32))]).reshape(-1, 1, 64)
    assert np.isfinite(x).all()
    c = kh.Cache(torch, [0], [len(x)], kv_heads=1, d=64, page=16, dtype="f32")
    c.append_new(x, x[::-1].copy())
    k, v = _read(c, [len(x)])
    assert np.array_equal(k, c.K[0]) and np.array_equal(v, c.V[0])


@pytest.mark.parametrize("d", [64, 128, 256])
def test_non_finite_rows_poison_their_token_and_head_only(torch, d):
    c = kh.Cache(torch, [5], [9], kv_heads=2, d=d, dtype="f32")
    k, v = c.rows(9), c.rows(9)
    k[1, 0, 3], v[2, 1, d - 1], k[4, 1, 40], v[4, 0, 0] = np.nan, np.inf, -np.inf, np.nan
    c.append_new(k, v)
    gk, gv = _read(c, [9])
    assert np.array_equal(gk, c.K[0][5:], equal_nan=True) and np.array_equal(gv, c.V[0][5:])
    assert np.isnan(gk).reshape(9, 2, d).all(-1).sum() == 4 and np.isnan(gk).any(-1).sum() == 4


def test_missing_pages_and_the_capacity(torch):
    """Rows of a page that is not there, or past the table, are dropped and read as zero."""
    past, new = [10, 40, 30], [60, 30, 2]
    c = kh.Cache(torch, past, new, d=64, spare=0, dtype="f32",
                 missing=[(0, 1, -1), (1, 3, 1 << 30), (2, 1, -7)])
    c.kv.length.copy_(torch.tensor(past, dtype=torch.int32))
    width = c.table.shape[1]
    before = _pools(c)
    n = [width * 16 + 20 - past[0], new[1], new[2]]  # sequence 0 runs past its table
    k, v = c.rows(sum(n)), c.rows(sum(n))
    c.append(n, k, v)
    ks, vs = okv.stored_pair(k, v)
    slots, there = [], np.zeros(sum(n), dtype=bool)
    for b, o in enumerate(kh.offsets(n)[:-1]):
        for i in range(n[b]):
            p = past[b] + i
            if p // 16 < width and 0 <= c.table[b, p // 16] < c.kv.k_codes.shape[1]:
                slots.append((b, p))
                there[o + i] = True
    _written(c, before, slots)
    gk, gv = _read(c, n)
    assert np.array_equal(gk[there], ks[there]) and np.array_equal(gv[there], vs[there])
    assert (gk[~there] == 0).all() and (gv[~there] == 0).all() and (~there).sum() > 20


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_commit_gathers_the_accepted_rows(torch, dtype):
    past, new = [0, 7, 30, 64, 5], [22, 6, 1, 40, 9]
    c = kh.Cache(torch, past, new, d=128, dtype=dtype, seed=9, layers=3, layer=1)
    k, v = c.append_new()
    rows = np.full((5, 24), -1, dtype=np.int32)
    picks = [[0, 2, 3, 21], [0, 1, 2, 3, 4, 5], [0], [0, 1, 9, 39, 39, 2], []]
    for b, p in enumerate(picks):
        rows[b, :len(p)] = p
    counts = np.array([4, 6, 3, 6, -2], dtype=np.int32)  # more than there are; negative
    rows[0, 1] = 77   # not a row of the sequence: slot left as it was
    before = _pools(c)
    length = c.kv.length.clone()
    new_length = torch.full((5,), -5, dtype=torch.int32, device="cuda")
    a = c.args(new, k=c.stack(k), v=c.stack(v))
    binding.kv_commit(a, kh.dev_i32(torch, rows), kh.dev_i32(torch, counts), new_length)
    torch.cuda.synchronize()
    assert torch.equal(c.kv.length, length)
    assert new_length.tolist() == [4, 13, 31, 70, 5]
    want = [[0, None, 3, 21], picks[1], picks[2], picks[3], []]
    slots, o = [], kh.offsets(new)
    ks, vs = okv.stored_pair(k, v)
    for b, p in enumerate(want):
        for i, r in enumerate(p):
            if r is not None:
                slots.append((b, past[b] + i))
                c.K[b][past[b] + i], c.V[b][past[b] + i] = ks[o[b] + r], vs[o[b] + r]
    _written(c, before, slots)
    gk, gv = _read(c, new)
    assert np.array_equal(gk, np.concatenate([c.K[b][past[b]:] for b in range(5)]))
    assert np.array_equal(gv, np.concatenate([c.V[b][past[b]:] for b in range(5)]))
    # in place and without rows: the lengths alone, held at the capacity
    cap = c.table.shape[1] * 16
    c.kv.length.copy_(torch.tensor([4, 13, 31, 70, cap - 1], dtype=torch.int32))
    before = _pools(c)
    binding.kv_commit(c.args(new), None, kh.dev_i32(torch, [1, 0, 5, 40, 9]), c.kv.length)
    torch.cuda.synchronize()
    assert c.kv.length.tolist() == [5, 13, 32, 110, cap]
    _written(c, before, [])


@pytest.mark.parametrize("where", ["apart", "in place", "over the counts"])
def test_commit_of_many_sequences_wherever_the_lengths_go(torch, where):
    S = 300
    past = [(7 * b) % 41 for b in range(S)]
    c = kh.Cache(torch, past, [2] * S, kv_heads=1, d=64, seed=3)
    k, v = c.append_new()
    rows = np.array([[1, 0, -1]] * S, dtype=np.int32)
    counts = np.array([b % 4 for b in range(S)], dtype=np.int32)
    cd = kh.dev_i32(torch, counts)
    new_length = {"apart": torch.full((S,), -5, dtype=torch.int32, device="cuda"),
                  "in place": c.kv.length, "over the counts": cd}[where]
    binding.kv_commit(c.args([2] * S, k=c.stack(k), v=c.stack(v)), kh.dev_i32(torch, rows), cd,
                      new_length)
    torch.cuda.synchronize()
    assert new_length.tolist() == [past[b] + min(b % 4, 2) for b in range(S)]
    ks, vs = okv.stored_pair(k, v)
    gk, gv = _read(c, [2] * S, begin=kh.dev_i32(torch, past))
    for b in range(S):
        for i, r in enumerate([1, 0]):
            r = r if i < b % 4 else i  # beyond the count: as appended
            assert np.array_equal(gk[2 * b + i], ks[2 * b + r])
            assert np.array_equal(gv[2 * b + i], vs[2 * b + r])


def test_append_on_another_stream_and_replayed(torch):
    """On a side stream, then captured in a graph and replayed with new rows and lengths."""
    c = kh.Cache(torch, [3, 50], [2, 1], d=128, dtype="bf16", spare=3)
    s = torch.cuda.Stream()
    k, v = c.rows(3), c.rows(3)
    kd, vd = c.stack(k), c.stack(v)
    a = c.args([2, 1], k=kd, v=vd)
    counts = kh.dev_i32(torch, [2, 1])
    s.wait_stream(torch.cuda.current_stream())
    binding.kv_append(a, stream=s)
    torch.cuda.synchronize()
    ks, vs = okv.stored_pair(k, v)
    gk, gv = _read(c, [2, 1])
    assert np.array_equal(gk, ks) and np.array_equal(gv, vs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.kv_append(a)
        binding.kv_commit(a, None, counts, c.kv.length)
    lengths = [3, 50]
    for step in range(4):
        k, v = c.rows(3), c.rows(3)
        kd.copy_(c.stack(k))
        vd.copy_(c.stack(v))
        g.replay()
        torch.cuda.synchronize()
        begin = kh.dev_i32(torch, lengths)
        gk, gv = _read(c, [2, 1], begin=begin)
        ks, vs = okv.stored_pair(k, v)
        assert np.array_equal(gk, ks) and np.array_equal(gv, vs)
        lengths = [lengths[0] + 2, lengths[1] + 1]
        assert c.kv.length.tolist() == lengths


def test_empty_batches_do_nothing(torch):
    c = kh.Cache(torch, [4], [0], d=64)
    before = _pools(c)
    c.append([0], c.rows(0), c.rows(0))
    _written(c, before, [])
    e = kh.Cache(torch, [], [], d=64)
    binding.kv_append(e.args([]))
