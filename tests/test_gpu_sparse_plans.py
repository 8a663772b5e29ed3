"""Sparse attention in the launches that long contexts take: units cut into equal parts, and the work line
with its join, for trees, for selections of several blocks whose last one is shorter, with two row tiles
and in fp32; selections whose rows do not fit LDS at once, over several chunks of pages; tables that are
full.  Every row is compared with attention in fp64 over the oracle's selection, within the bound of
kv_harness; the oracle is written as matrix products here, since the sizes are those of real calls."""
import numpy as np
import pytest

from gated_deltanet_tree_amd import binding

import kv_harness as kh
import sparse_harness as sh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    binding.lib()
    return torch


def _cache(torch, past, new, **kw):
    c = sh.SparseCache(torch, past, new, **kw)
    c.append_new()
    c.build_bounds()
    return c


def _selections(c, b, q, top, share, first, last):
    """As oracle.sparse.select with every page there: [selections][Hkv, min(top, full)]."""
    page, full = c.page, c.past[b] // c.page
    G = q.shape[1] // c.H
    K = c.K[b][:full * page].reshape(full, page, c.H, c.d)
    hi, lo = K.max(1), K.min(1)
    out = []
    for i0, i1 in sh.osp.selections(len(q), share):
        sel = np.zeros((c.H, min(top, full)), dtype=np.int64)
        for h in range(c.H):
            if full <= top:
                sel[h] = np.arange(full)
                continue
            rows = q[i0:i1, h * G:(h + 1) * G].reshape(-1, c.d)
            score = (np.maximum(rows, 0) @ hi[:, h].T + np.minimum(rows, 0) @ lo[:, h].T).max(0)
            rest = np.arange(first, full - last)
            best = rest[np.argsort(-score[rest], kind="stable")[:top - first - last]]
            sel[h] = np.sort(np.concatenate([np.arange(first), best, np.arange(full - last, full)]))
        out.append(sel)
    return out


def _check(torch, c, q, sel, out, top, share, first=1, last=1, trees=None, weight_half=2.0 ** -8):
    """Selections equal; outputs within kv_harness.check_rows' bound, computed in fp64 on the device."""
    scale, f64 = c.d ** -0.5, dict(dtype=torch.float64, device="cuda")
    half, out_half = (weight_half, 2.0 ** -8) if c.dtype == "bf16" else (0.0, 3 * kh.U)
    for b, o in enumerate(kh.offsets(c.new)[:-1]):
        n, full = c.new[b], c.past[b] // c.page
        if n == 0:
            continue
        G = q.shape[1] // c.H
        see = c.visible(b, trees)
        want = _selections(c, b, q[o:o + n], top, share, first, last)
        K, V = torch.tensor(c.K[b], **f64), torch.tensor(c.V[b], **f64)
        for g, (i0, i1) in enumerate(sh.osp.selections(n, share)):
            k = min(top, full)
            assert np.array_equal(sel[o + i0, :, :k], want[g]), (b, g)
            assert (sel[o + i0, :, k:] == -1).all()
            for h in range(c.H):
                part = sh.osp.visible(see[i0:i1], want[g][h], c.page, full)
                at = np.flatnonzero(part.any(0))
                mask = torch.tensor(np.repeat(part[:, at], G, 0), device="cuda")
                kk, vv = K[torch.tensor(at), h], V[torch.tensor(at), h]
                rows = torch.tensor(q[o + i0:o + i1, h * G:(h + 1) * G].reshape(-1, c.d), **f64)
                got = torch.tensor(out[o + i0:o + i1, h * G:(h + 1) * G].reshape(-1, c.d), **f64)
                kt = kk.T.contiguous()
                w = torch.softmax((scale * (rows @ kt)).masked_fill(~mask, -torch.inf), -1)
                ref, mag = w @ vv, w @ vv.abs()
                size = scale * (rows.abs() @ kt.abs()).masked_fill(~mask, 0.0).amax(-1)
                eps = 2 * ((c.d + 8) * kh.U * size + 4 * kh.U * size + 4 * kh.U) + (mask.sum(-1) + 8) * kh.U
                bound = (eps + half)[:, None] * (mag + ref.abs()) + out_half * ref.abs() + 1e-30
                worst = ((got - ref).abs() / bound).amax().item()
                assert worst <= 1.0, (b, g, h, worst)  # a NaN fails too


def _run(torch, c, heads, top, share, plan, trees=None, max_length=0):
    """plan: 'line' or 'parts', which the launch has to be; the rest as select_and_attend."""
    a = c.args(c.new, q=torch.empty((c.layers, sum(c.new), heads, c.d), device="cuda",
                                    dtype=torch.bfloat16 if c.dtype == "bf16" else torch.float32), max_length=max_length)
    need = binding.sparse_workspace_bytes(a, binding.sparse_args(a, c.bounds, None, top, share, 1, 1))
    G = heads // c.H
    tokens = min(share or max(c.new), max(c.new))
    tile = 64 if c.dtype == "bf16" and c.d <= 128 and tokens * G > 32 else 32
    blocks = max(sum(-(-(i1 - i0) * G // tile) for i0, i1 in sh.osp.selections(n, share)) for n in c.new)
    units, each = blocks * len(c.new) * c.H, 2 * tile * (c.d + 2) * 4
    groups, rest = divmod(need - 8 * units, each)
    assert rest == 0, "the selection needs more workspace than the attention"
    slots = 512 if tile == 64 or c.d > 64 else 768
    if plan == "line":
        assert groups == slots and groups % units != 0
    else:
        assert groups % units == 0 and groups > units
    q, sel, out = c.select_and_attend(heads, top, share=share, first=1, last=1, trees=trees, max_length=max_length)
    _check(torch, c, q, sel, out, top, share, trees=trees)
    again = c.select_and_attend(heads, top, share=share, first=1, last=1, trees=trees, max_length=max_length, q=q)
    assert np.array_equal(sel, again[1]) and np.array_equal(out, again[2])


SHORT = [100, 900, 30, 2000, 64, 63, 700, 128, 1500, 5]


@pytest.mark.parametrize("dtype,d,page,top,kv_heads", [("bf16", 128, 64, 100, 4), ("bf16", 64, 64, 100, 4),
                                                       ("bf16", 256, 64, 70, 2), ("f32", 128, 64, 100, 2),
                                                       ("f32", 256, 128, 60, 2)])
def test_trees_on_the_line(torch, dtype, d, page, top, kv_heads):
    """Trees of 1 to 64 nodes, six query heads a kv head, on two long caches and many short ones."""
    rng = np.random.default_rng(d)
    sizes = [22, 33, 22, 1, 22, 64, 22, 2, 22, 22, 7, 22]
    trees = [kh.random_tree(rng, n, 4, 20) for n in sizes]
    c = _cache(torch, [(top + 9) * page + 11, (top + 2) * page] + SHORT, sizes, kv_heads=kv_heads, d=d, dtype=dtype,
               page=page)
    _run(torch, c, 6 * kv_heads, top, 0, "line", trees)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 256), ("f32", 128), ("f32", 256)])
def test_chunks_on_the_line(torch, dtype, d):
    """Sixteen tokens a selection, one block of rows each, the last ones shorter."""
    c = _cache(torch, [66 * 64 + 1, 58 * 64 + 63, 200, 2000], [700, 330, 1, 177], kv_heads=4, d=d, dtype=dtype, page=64)
    _run(torch, c, 16 if dtype == "bf16" and d < 256 else 8, 55, 16, "line")


@pytest.mark.parametrize("dtype,d,share,kv_heads,heads", [("bf16", 128, 64, 4, 24), ("bf16", 128, 31, 4, 64),
                                                          ("f32", 128, 64, 2, 12), ("bf16", 64, 50, 4, 40)])
def test_selections_of_several_blocks_on_the_line(torch, dtype, d, share, kv_heads, heads):
    """The last selection of a sequence has one token, or a few, and fewer blocks than the others."""
    c = _cache(torch, [99 * 64 + 5, 96 * 64, 300, 7], [3 * share + 1, share + 1, share + 6, 3],
               kv_heads=kv_heads, d=d, dtype=dtype, page=64)
    _run(torch, c, heads, 94, share, "line")


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 128), ("f32", 256)])
@pytest.mark.parametrize("tree", [True, False])
def test_units_cut_into_equal_parts(torch, dtype, d, tree):
    """One long cache beside a short one: every unit is joined from many fragments."""
    trees = [kh.random_tree(np.random.default_rng(1), n, 4, 20) for n in (22, 9)] if tree else None
    c = _cache(torch, [5000, 70], [22, 9], kv_heads=2, d=d, dtype=dtype, page=64)
    _run(torch, c, 12, 60, 0, "parts", trees)


@pytest.mark.parametrize("dtype,past,new,kv_heads,heads,share", [
    ("bf16", [16 * 1800 + 3], [60], 1, 5, 0),      # 300 rows, 256 at a time, two chunks of pages
    ("f32", [16 * 1800 + 3], [45], 1, 5, 0),       # 225 rows, 144 at a time
    ("f32", [16 * 750, 16 * 20], [260, 3], 4, 20, 16)])  # more selections than compute units, 80 rows each
def test_rows_that_do_not_fit_at_once_over_several_chunks_of_pages(torch, dtype, past, new, kv_heads, heads, share):
    """The rows are laid out again for every chunk; a short expected length keeps it in one share."""
    c = _cache(torch, past, new, kv_heads=kv_heads, d=64, dtype=dtype, page=16)
    q, sel, out = c.select_and_attend(heads, 9, share=share, first=1, last=1, max_length=100)
    _check(torch, c, q, sel, out, 9, share)


def test_full_tables_and_lengths_outside_them(torch):
    """Four pages, all of them written.  A length past the table is the table's: the new token sees the two
    pages of its selection; a length below zero is zero: it sees slot 0 only."""
    c = _cache(torch, [63, 63], [1, 1], page=16, spare=0)
    c.kv.length.copy_(torch.tensor([10**9, -5], dtype=torch.int32))
    c.bounds.fill_(77.0)
    a = c.args([64, 0])
    binding.kv_bounds(a, binding.sparse_args(a, c.bounds))
    q, sel, out = c.select_and_attend(4, 2)
    want = sh.osp.select(q[:1], c.K[0], 16, 4, 2)[0]
    assert np.array_equal(sel[0], want) and (sel[1] == -1).all()
    for h in range(2):
        rows = slice(2 * h, 2 * h + 2)
        see = np.zeros((1, 64), dtype=bool)
        for e in want[h]:
            see[0, 16 * e:16 * e + 16] = True
        kh.check_rows(q[:1, rows], out[:1, rows], c.K[0][:, h:h + 1], c.V[0][:, h:h + 1], see, 128 ** -0.5, "bf16")
        one = np.arange(64)[None] == 0
        kh.check_rows(q[1:, rows], out[1:, rows], c.K[1][:, h:h + 1], c.V[1][:, h:h + 1], one, 128 ** -0.5, "bf16")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group,share,new", [(1, 1, 5), (4, 4, 9), (16, 1, 3), (3, 5, 11), (2, 0, 8)])
def test_up_to_16_rows_a_selection_keep_what_rounding_leaves_of_the_weights(torch, d, group, share, new):
    """A weight enters as its rounding and the rounding of the rest, off by 2^-8 of 2^-8 of it: as the
    dense calls, whole and cut over workgroups, with flat and with peaked scores."""
    past, news = [2300, 0, 61], [new, max(new - 1, 1), 1]
    c = _cache(torch, past, news, kv_heads=2, d=d, page=32)
    for q_scale in (1.0, 4.0):
        for top in (4, 60):
            q, sel, out = c.select_and_attend(2 * group, top, share=share, first=1, last=1, q_scale=q_scale)
            _check(torch, c, q, sel, out, top, share, weight_half=2.0 ** -16)


def test_two_captured_calls_replayed_at_once(torch):
    """Selection in shares and attention in parts or on the line, with workspaces of their own, on two streams, with
    eager work between: every replay gives what the eager calls gave."""
    calls = []
    for past, new, kv_heads, heads, top, share in (([9000], [1], 2, 8, 40, 1),
                                                   ([5000, 3000], [300, 270], 4, 16, 40, 16)):
        c = _cache(torch, past, new, kv_heads=kv_heads, d=128, page=64, seed=len(past))
        q = kh.to_dev(torch, kh.rng_rows(c.rng, (1, sum(new), heads, 128), "bf16", 1.5), "bf16")
        out = torch.empty_like(q)
        sel = torch.full((1, sum(new), kv_heads, top), -7, dtype=torch.int32, device="cuda")
        sparse = lambda a: binding.sparse_args(a, c.bounds, sel, top, share, 1, 1)  # noqa: E731
        need = binding.sparse_workspace_bytes(c.args(new, q=q, out=out), sparse(c.args(new, q=q, out=out)))
        assert need > 0
        a = c.args(new, q=q, out=out, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
        x = sparse(a)
        binding.kv_select(a, x)
        binding.sparse_attention(a, x)
        torch.cuda.synchronize()
        want = (sel.clone(), out.clone())
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph):
            binding.kv_select(a, x)
            binding.sparse_attention(a, x)
        calls.append((graph, side, a, x, sel, out, want, c))
    for i in range(6):
        for graph, side, a, x, sel, out, want, c in calls:
            sel.fill_(-7)
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        for graph, side, *rest in calls:
            with torch.cuda.stream(side):
                for _ in range(i + 1):
                    graph.replay()
        torch.cuda.synchronize()
        for graph, side, a, x, sel, out, want, c in calls:
            assert torch.equal(sel, want[0]) and torch.equal(out, want[1]), i
