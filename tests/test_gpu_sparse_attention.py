"""Page bounds, page selections and sparse attention over the 4-bit cache against the oracle."""
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


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_bounds_of_the_full_pages_and_no_others(torch, d, page):
    c = _cache(torch, [0, page - 1, page, 5 * page + 3, 700], [1, 1, 0, 2, 3], d=d, page=page, kv_heads=2, layers=2,
               layer=1, missing=[(3, 2, -1), (4, 0, 10**6)])
    c.check_bounds()


def test_bounds_after_a_commit_are_those_of_the_pages_it_filled(torch):
    """Twenty committed tokens over pages of 16: what an earlier call wrote stays."""
    c = _cache(torch, [40, 16, 3, 64], [1, 1, 1, 1], page=16)
    before = kh.host(c.bounds)
    mark = c.bounds.clone().fill_(-5.0)
    a = c.args([20, 0, 2, 64])
    binding.kv_bounds(a, binding.sparse_args(a, mark))
    got = kh.host(mark)
    # slots 20 .. 39 touch pages 1 and 2, of which 1 is full; none; none full; all four
    touched = {(0, 1)} | {(3, i) for i in range(4)}
    want = np.full(got.shape, -5.0)
    for b, i in touched:
        want[0, c.table[b, i]] = before[0, c.table[b, i]]
    assert np.array_equal(got, want)


def test_a_key_that_is_not_finite_shows_in_its_heads_bounds(torch):
    c = sh.SparseCache(torch, [0], [40], d=128, page=16, kv_heads=2)
    k, v = c.rows(40), c.rows(40)
    k[5, 0, 100], v[20, 1, 3] = np.inf, np.nan
    c.append_new(k, v)
    c.kv.length.fill_(40)
    c.past, c.new = [40], [0]
    c.build_bounds()
    got = kh.host(c.bounds)[0, c.table[0, :2]]
    nan = np.isnan(got).any((-1, -2))
    assert nan.tolist() == [[True, False], [False, True]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 4, 6, 16, 20])
def test_single_tokens(torch, d, dtype, group):
    """One new token a sequence, from no full page to many; one sequence without any."""
    c = _cache(torch, [0, 5, 16, 80, 95, 96, 97, 333, 150], [1] * 8 + [0], kv_heads=2, d=d, dtype=dtype, seed=group,
               page=16)
    for top, first, last in ((1, 0, 0), (5, 1, 1), (3, 2, 1), (64, 1, 0)):
        q, sel, out = c.select_and_attend(2 * group, top, first=first, last=last)
        c.check_sparse(q, sel, out, top, first=first, last=last)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,page", [(64, 32), (128, 64), (256, 16)])
@pytest.mark.parametrize("share", [1, 3, 16, 0])
def test_tokens_that_share_a_selection(torch, d, dtype, page, share):
    """Ragged chunks of prompts: selections of 1, 3, 16 tokens and of all, the last ones shorter."""
    c = _cache(torch, [6 * page + 5, 0, 9 * page, page - 1], [35, 20, 1, 17], kv_heads=2, d=d, dtype=dtype, page=page,
               layers=2, layer=1, seed=share)
    q, sel, out = c.select_and_attend(12, 4, share=share, first=1, last=1)
    c.check_sparse(q, sel, out, 4, share=share, first=1, last=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_trees(torch, d, dtype):
    rng = np.random.default_rng(d)
    sizes = [1, 2, 7, 22, 64, 33]
    trees = [kh.random_tree(rng, n, 4, 20) for n in sizes]
    c = _cache(torch, [3, 64, 130, 300, 77, 16], sizes, kv_heads=2, d=d, dtype=dtype, page=16)
    q, sel, out = c.select_and_attend(6, 4, share=0, first=1, last=1, trees=trees)
    c.check_sparse(q, sel, out, 4, share=0, first=1, last=1, trees=trees)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("max_length", [0, 1, 40, 2000, 20000])
def test_pages_split_over_workgroups(torch, dtype, max_length):
    """More pages than a workgroup holds at once, in one share and in several; repeatable bit for bit."""
    c = _cache(torch, [18000, 1000], [2, 1], kv_heads=1, d=64, dtype=dtype, page=16)
    for top in (7, 256):
        q, sel, out = c.select_and_attend(4, top, first=1, last=2, max_length=max_length)
        c.check_sparse(q, sel, out, top, first=1, last=2)
        again = c.select_and_attend(4, top, first=1, last=2, max_length=max_length, q=q)
        assert np.array_equal(sel, again[1]) and np.array_equal(out, again[2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("expected,full", [(300, 299), (300, 302), (300, 303), (300, 600), (2052, 2050), (2052, 2051),
                                           (2052, 2053)])
def test_shares_with_more_pages_than_expected(torch, dtype, expected, full):
    """All pages of the shares fit the join, or only the best of each do: more than `expected`, or than 2048."""
    c = _cache(torch, [16 * full + 5, 16 * 7], [1, 1], kv_heads=1, d=256, page=16, spare=3, dtype=dtype)
    for top in (5, 60):
        q, sel, out = c.select_and_attend(4, top, first=1, last=1, max_length=16 * expected)
        c.check_sparse(q, sel, out, top, first=1, last=1)


def test_many_rows_share_a_selection_over_many_pages(torch):
    """Several tiles of rows over several chunks of pages."""
    c = _cache(torch, [17500], [40], kv_heads=1, d=64, page=16)
    q, sel, out = c.select_and_attend(5, 9, share=0, first=1, last=1, max_length=100)
    c.check_sparse(q, sel, out, 9, share=0, first=1, last=1)


@pytest.mark.parametrize("splits", [0, 50])
def test_equal_pages_are_taken_in_order(torch, splits):
    c = sh.SparseCache(torch, [16 * 300 + 2], [1], kv_heads=1, d=64, page=16)
    one = c.rows(16)
    k = np.concatenate([np.tile(one, (300, 1, 1)), c.rows(2)])
    c.kv.length.zero_()
    c.append([16 * 300 + 2], k, k)
    c.kv.length.fill_(16 * 300 + 2)
    ks = np.array(sh.okv.stored_pair(k, k))
    c.K[0][:4802], c.V[0][:4802] = ks
    c.append_new()
    c.build_bounds()
    q, sel, out = c.select_and_attend(4, 20, first=2, last=3, max_length=splits)
    assert sel[0, 0].tolist() == list(range(17)) + [297, 298, 299]
    c.check_sparse(q, sel, out, 20, first=2, last=3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("near", [2, 5, 40])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_pages_nearer_than_32_bits_resolve(torch, d, dtype, near):
    """Pages that differ by 2^-22 in one channel, of sums in the hundreds: the larger one is taken, and the
    lower among equals.  A few of them, or most, among pages that are far below; in one share (a short expected
    length) and in several."""
    c = sh.SparseCache(torch, [60 * 16], [2], kv_heads=2, d=d, page=16, dtype=dtype, spare=6000)
    one = np.abs(c.rows(1))
    k = np.tile(0.125 * one, (960, 1, 1))
    k[:, :, d - 32:] = 0.0
    who = np.sort(c.rng.permutation(60)[:near])
    for n, page in enumerate(who):
        k[16 * page:16 * page + 16] = one
        k[16 * page:16 * page + 16, :, d - 32:] = 0.0
        k[16 * page + n % 16, :, d - 1] = 2.0 ** -22 * [1, 3, 0.5, 3, 2, 1.5][n % 6]
    c.kv.length.zero_()
    c.append([960], k, k)
    c.kv.length.fill_(960)
    c.K[0][:960], c.V[0][:960] = sh.okv.stored_pair(k, k)
    c.append_new()
    c.build_bounds()
    q = np.abs(kh.rng_rows(c.rng, (2, 6, d), dtype, 4.0)) + 1.0
    q[..., d - 1] = 1.0
    q = kh.host(kh.to_dev(torch, q, dtype))  # as the kernel gets them
    for top in {1, near // 2, near - 1, near, min(near + 3, 59)}:
        for max_length in (0, 64):
            q, sel, out = c.select_and_attend(6, top, share=0, q=q, max_length=max_length)
            c.check_sparse(q, sel, out, top, share=0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pages_that_are_not_there_come_last(torch, dtype):
    c = _cache(torch, [170, 90], [1, 2], page=16, dtype=dtype, spare=0,
               missing=[(0, 0, -1), (0, 5, 10**9), (0, 9, -3), (1, 1, -1), (1, 2, -1), (1, 3, -1), (1, 4, -1)])
    for top in (4, 9):
        q, sel, out = c.select_and_attend(4, top, share=0, last=1)
        c.check_sparse(q, sel, out, top, share=0, last=1)


def test_a_row_that_sees_nothing_is_zero(torch):
    """Every page of the sequence is missing."""
    c = _cache(torch, [50], [1], page=16, spare=0, missing=[(0, i, -1) for i in range(4)])
    q, sel, out = c.select_and_attend(4, 2)
    assert sel[0, 0].tolist() == [0, 1] and not out.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_queries_that_are_not_finite(torch, dtype):
    """Their rows are NaN; the rows that share their selection are not touched by them."""
    c = _cache(torch, [200, 200], [3, 3], page=16, dtype=dtype, kv_heads=1)
    q = kh.rng_rows(c.rng, (6, 4, 128), dtype, 1.5)
    q[1, 2, 5], q[2, 0, 0] = np.nan, np.inf
    q[3:, :, 7] = -np.inf
    q, sel, out = c.select_and_attend(4, 5, share=0, first=1, q=q)
    bad = ~np.isfinite(q).all(-1)
    assert np.isnan(out[bad]).all() and np.isfinite(out[~bad]).all()
    clean = np.where(bad[..., None], 0.0, q)
    want = sh.osp.select(q[:3], c.K[0], 16, 12, 5, 0, 1)
    assert np.array_equal(sel[0], want[0])
    assert sel[3, 0].tolist() == [0, 1, 2, 3, 4]
    part = sh.osp.visible(c.visible(0), want[0][0], 16, 12)
    got = np.where(bad[..., None], 0.0, out)[:3]
    ref = sh.okv.attention(clean[:3], c.K[0], c.V[0], part, 128 ** -0.5)
    keep = ~bad[:3]
    assert np.abs(got - ref)[keep].max() < 0.02 * np.abs(ref).max()


def test_a_poisoned_page_is_selected_and_shows(torch):
    c = sh.SparseCache(torch, [0], [200], page=16, kv_heads=2)
    k, v = c.rows(200), c.rows(200)
    k[37, 1, 9] = np.nan
    c.append_new(k, v)
    c.kv.length.fill_(199)
    c.past, c.new = [199], [1]
    c.build_bounds()
    q, sel, out = c.select_and_attend(4, 3, first=1, last=1)
    assert sel[0, 1].tolist() == [0, 2, 11]
    assert np.isfinite(out[0, :2]).all() and np.isnan(out[0, 2:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_selections_of_the_callers_own(torch, dtype):
    """The attention takes any: entries outside the full pages are dropped, -1 and others."""
    c = _cache(torch, [167, 40, 3], [2, 1, 1], page=16, dtype=dtype)
    own = np.array([[[9, 1, 4], [-1, 3, 10]], [[2, 0, 5], [0, 1, 2]], [[-5, 2**31 - 1, 0], [1, -2**31, 1000]],
                    [[0, 1, 2], [3, 4, 5]]])
    q, sel, out = c.select_and_attend(6, 3, selected=own)
    c.check_sparse(q, sel, out, 3, chosen=own)


def test_few_pages_are_dense_attention(torch):
    """With no more full pages than a selection holds, the rows see what the dense call lets them."""
    c = _cache(torch, [100, 30, 0], [3, 1, 2], page=16)
    q, sel, out = c.select_and_attend(4, 8, first=1)
    _, dense = c.attend(4, q=q)
    c.check(q, out)
    assert np.abs(out - dense).max() <= 2 ** -7 * np.abs(dense).max()


def test_lengths_past_the_capacity_and_below_zero(torch):
    """Tables of four pages, every slot of them written."""
    c = _cache(torch, [63, 63], [1, 1], page=16, spare=0)
    c.kv.length.copy_(torch.tensor([10**9, -5], dtype=torch.int32))
    cap = c.table.shape[1] * 16
    c.K = [np.concatenate([k, np.zeros((cap + 1 - len(k), 2, 128))]) for k in c.K]
    q, sel, out = c.select_and_attend(4, 2)
    full = cap // 16
    assert set(sel[0].flatten()) <= set(range(full)) and (sel[1] == -1).all()
    assert np.isfinite(out).all()


@pytest.mark.parametrize("d", [64, 128])
def test_many_selections(torch, d):
    """Enough of them to fill the device whole, and more rows a selection than a tile holds."""
    c = _cache(torch, [700, 100, 350], [300, 2, 77], kv_heads=2, d=d, page=32)
    for share in (1, 7):
        q, sel, out = c.select_and_attend(32, 5, share=share, first=1, last=1)
        c.check_sparse(q, sel, out, 5, share=share, first=1, last=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_selections_over_many_pages(torch, dtype):
    """More selections than the device has compute units, of more pages than a workgroup holds at once."""
    c = _cache(torch, [16 * 1500 + 3, 16 * 900], [270, 3], kv_heads=1, d=64, page=16, dtype=dtype)
    for top in (6, 256):
        q, sel, out = c.select_and_attend(2, top, first=1, last=1)
        c.check_sparse(q, sel, out, top, first=1, last=1)


@pytest.mark.parametrize("max_length", [0, 64])
def test_many_selections_of_equal_pages(torch, max_length):
    """More selections than the device has compute units, every page in doubt."""
    c = sh.SparseCache(torch, [960], [300], kv_heads=1, d=64, page=16)
    k = np.tile(c.rows(1), (960, 1, 1))
    c.kv.length.zero_()
    c.append([960], k, k)
    c.kv.length.fill_(960)
    c.K[0][:960], c.V[0][:960] = sh.okv.stored_pair(k, k)
    c.append_new()
    c.build_bounds()
    q, sel, out = c.select_and_attend(2, 9, first=1, last=2, max_length=max_length)
    assert (sel[:, 0] == [0, 1, 2, 3, 4, 5, 6, 58, 59]).all()
    c.check_sparse(q, sel, out, 9, first=1, last=2)


def test_several_layers_in_one_call(torch):
    """Bounds, selection and attention of two layers at once, each as alone."""
    S, H, d, page, top = 3, 2, 128, 16, 3
    past, new, G = [100, 17, 64], [2, 1, 3], 3
    rng = np.random.default_rng(12)
    kv = binding.alloc_kv_cache(2, S, H, d, 40, page, 9)
    kv.pages.copy_(torch.from_numpy(rng.permutation(40)[:27].reshape(3, 9).astype(np.int32)))
    offs, dev = kh.offsets(past), kh.dev_i32(torch, kh.offsets(past))
    k, v = (kh.rng_rows(rng, (2, sum(past), H, d), "bf16") for _ in range(2))
    a = binding.kv_args(kv, offs, dev, k=kh.to_dev(torch, k, "bf16"), v=kh.to_dev(torch, v, "bf16"), n_layers=2)
    binding.kv_append(a)
    binding.kv_commit(a, None, kh.dev_i32(torch, past), kv.length)
    bounds = binding.alloc_kv_bounds(kv)
    binding.kv_bounds(a, binding.sparse_args(a, bounds))
    no, nd, T = kh.offsets(new), kh.dev_i32(torch, kh.offsets(new)), sum(new)
    kn, vn = (kh.rng_rows(rng, (2, T, H, d), "bf16") for _ in range(2))
    q = kh.rng_rows(rng, (2, T, H * G, d), "bf16", 1.5)
    qd = kh.to_dev(torch, q, "bf16")
    out, sel = torch.full_like(qd, float("nan")), torch.full((2, T, H, top), -7, dtype=torch.int32, device="cuda")
    kw = dict(q=qd, out=out, k=kh.to_dev(torch, kn, "bf16"), v=kh.to_dev(torch, vn, "bf16"), n_layers=2)

    def sparse(x):
        return binding.sparse_args(x, bounds, sel, top, 0, 1, 1)

    x = binding.kv_args(kv, no, nd, **kw)
    ws = torch.empty(binding.sparse_workspace_bytes(x, sparse(x)) + 16, dtype=torch.uint8, device="cuda")
    x = binding.kv_args(kv, no, nd, workspace=ws, **kw)
    binding.kv_append(x)
    binding.kv_select(x, sparse(x))
    binding.sparse_attention(x, sparse(x))
    torch.cuda.synchronize()
    got, chosen = kh.host(out), sel.cpu().numpy()
    for l in range(2):
        for b in range(S):
            ks, vs = sh.okv.stored_pair(k[l, offs[b]:offs[b + 1]], v[l, offs[b]:offs[b + 1]])
            kt, vt = sh.okv.stored_pair(kn[l, no[b]:no[b + 1]], vn[l, no[b]:no[b + 1]])
            K, V, full = np.concatenate([ks, kt]), np.concatenate([vs, vt]), past[b] // page
            sl = slice(no[b], no[b + 1])
            want = sh.osp.select(q[l, sl], K, page, full, top, 0, 1, 1)[0]
            assert np.array_equal(chosen[l, no[b], :, :min(top, full)], want)
            see = sh.okv.visible_causal(past[b], new[b])
            for h in range(H):
                c = slice(h * G, (h + 1) * G)
                kh.check_rows(q[l, sl][:, c], got[l, sl][:, c], K[:, h:h + 1], V[:, h:h + 1],
                              sh.osp.visible(see, want[h], page, full), d ** -0.5, "bf16")


def test_pages_and_limits_past_4_gib(torch):
    """The last pages of a pool whose limits alone take more than 4 GiB."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GiB")
    n_pages, page, d, past = (1 << 24) + 5000, 16, 64, 16 * 30 + 3
    kv = binding.alloc_kv_cache(1, 1, 1, d, n_pages, page, 32)
    rng = np.random.default_rng(13)
    kv.pages.copy_(torch.from_numpy((n_pages - 1 - rng.permutation(4000)[:32]).astype(np.int32)[None]))
    bounds = torch.empty((1, n_pages, 1, 2, d), dtype=torch.bfloat16, device="cuda")
    assert bounds.numel() * 2 > 1 << 32
    offs = np.array([0, past], dtype=np.int32)
    k, v = (kh.rng_rows(rng, (1, past, 1, d), "bf16") for _ in range(2))
    a = binding.kv_args(kv, offs, kh.dev_i32(torch, offs), k=kh.to_dev(torch, k, "bf16"), v=kh.to_dev(torch, v, "bf16"))
    binding.kv_append(a)
    binding.kv_commit(a, None, kh.dev_i32(torch, [past]), kv.length)
    binding.kv_bounds(a, binding.sparse_args(a, bounds))
    one = np.array([0, 1], dtype=np.int32)
    kn, vn = (kh.rng_rows(rng, (1, 1, 1, d), "bf16") for _ in range(2))
    q = kh.rng_rows(rng, (1, 1, 4, d), "bf16", 1.5)
    qd = kh.to_dev(torch, q, "bf16")
    out, sel = torch.empty_like(qd), torch.full((1, 1, 1, 5), -7, dtype=torch.int32, device="cuda")
    kw = dict(q=qd, out=out, k=kh.to_dev(torch, kn, "bf16"), v=kh.to_dev(torch, vn, "bf16"))
    x = binding.kv_args(kv, one, kh.dev_i32(torch, one), **kw)
    sp = binding.sparse_args(x, bounds, sel, 5)
    ws = torch.empty(binding.sparse_workspace_bytes(x, sp) + 16, dtype=torch.uint8, device="cuda")
    x = binding.kv_args(kv, one, kh.dev_i32(torch, one), workspace=ws, **kw)
    binding.kv_append(x)
    binding.kv_select(x, sp)
    binding.sparse_attention(x, sp)
    torch.cuda.synchronize()
    ks, vs = sh.okv.stored_pair(np.concatenate([k[0], kn[0]]), np.concatenate([v[0], vn[0]]))
    want = sh.osp.select(q[0], ks, page, 30, 5)[0]
    assert np.array_equal(sel[0, 0].cpu().numpy(), want)
    see = sh.osp.visible(sh.okv.visible_causal(past, 1), want[0], page, 30)
    kh.check_rows(q[0], kh.host(out[0]), ks, vs, see, d ** -0.5, "bf16")


def test_another_stream(torch):
    c = _cache(torch, [500], [4], page=16)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    q, sel, out = c.select_and_attend(4, 6, stream=s)
    c.check_sparse(q, sel, out, 6)


def test_captured_steps_while_the_cache_grows(torch):
    """One captured step (append, select, attend, commit, bounds) replayed: the selection follows the
    lengths it finds, and the bounds keep up."""
    S, H, d, page, top, steps = 2, 1, 64, 16, 3, 70
    rng = np.random.default_rng(5)
    kv = binding.alloc_kv_cache(1, S, H, d, 12, page, 6)
    kv.pages.copy_(torch.from_numpy(rng.permutation(12).reshape(2, 6).astype(np.int32)))
    kv.length.copy_(torch.tensor([0, 21], dtype=torch.int32))
    past = [0, 21]
    offs = np.arange(S + 1, dtype=np.int32)
    dev_offs = kh.dev_i32(torch, offs)
    f = dict(dtype=torch.bfloat16, device="cuda")
    k, v, q, out = (torch.zeros((1, S, h, d), **f) for h in (H, H, 4, 4))
    bounds = binding.alloc_kv_bounds(kv)
    sel = torch.full((1, S, H, top), -1, dtype=torch.int32, device="cuda")
    hist = [[np.zeros((0, H, d))] * 2 for _ in range(S)]
    first = kh.rng_rows(rng, (2, 21, H, d), "bf16")
    fill = kh.offsets([0, 21])
    kv.length.zero_()
    a0 = binding.kv_args(kv, fill, kh.dev_i32(torch, fill), k=kh.to_dev(torch, first[:1], "bf16"),
                         v=kh.to_dev(torch, first[1:], "bf16"))
    binding.kv_append(a0)
    binding.kv_commit(a0, None, kh.dev_i32(torch, [0, 21]), kv.length)
    binding.kv_bounds(a0, binding.sparse_args(a0, bounds))
    hist[1] = list(sh.okv.stored_pair(first[0], first[1]))
    a = binding.kv_args(kv, offs, dev_offs, q=q, k=k, v=v, out=out)
    need = binding.sparse_workspace_bytes(a, binding.sparse_args(a, bounds, sel, top, keep_last=1))
    ws = torch.zeros(need + 16, dtype=torch.uint8, device="cuda")
    a = binding.kv_args(kv, offs, dev_offs, q=q, k=k, v=v, out=out, workspace=ws)
    x = binding.sparse_args(a, bounds, sel, top, keep_last=1)
    ones = torch.ones(S, dtype=torch.int32, device="cuda")

    def step():
        binding.kv_append(a)
        binding.kv_select(a, x)
        binding.sparse_attention(a, x)
        binding.kv_commit(a, None, ones, kv.length)
        binding.kv_bounds(a, x)

    saved = {n: t.clone() for n, t in (("length", kv.length), ("bounds", bounds))}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    kv.length.copy_(saved["length"])
    bounds.copy_(saved["bounds"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        ki, vi = (kh.rng_rows(rng, (S, H, d), "bf16") for _ in range(2))
        qi = kh.rng_rows(rng, (S, 4, d), "bf16", 1.5)
        for t, y in ((k, ki), (v, vi), (q, qi)):
            t.copy_(kh.to_dev(torch, y[None], "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        ks, vs = sh.okv.stored_pair(ki, vi)
        got, chosen = kh.host(out[0]), sel[0].cpu().numpy()
        for b in range(S):
            hist[b] = [np.concatenate([hist[b][0], ks[b:b + 1]]), np.concatenate([hist[b][1], vs[b:b + 1]])]
            full = past[b] // page
            want = sh.osp.select(qi[b:b + 1], hist[b][0], page, full, top, 1, 0, 1)[0]
            m = min(top, full)
            assert np.array_equal(chosen[b, :, :m], want) and (chosen[b, :, m:] == -1).all(), (i, b)
            see = sh.okv.visible_causal(past[b], 1)
            kh.check_rows(qi[b:b + 1], got[b:b + 1], hist[b][0], hist[b][1],
                          sh.osp.visible(see, want[0], page, full), d ** -0.5, "bf16")
            past[b] += 1
    assert past[1] // page > top
