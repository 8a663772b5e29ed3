"""Log probabilities of rows of logits against the oracle.

Bound, with u = 2^-24, p the oracle's probabilities, a_j = m - l_j and D = sum p a:
  a weight's exponent is off by 3 u a (difference, factor, product), exp2 by 2 u, a piece's sum of 32
  terms in four chains and over 64 lanes by 16 u more:   |d log Z| <= u (3 D + 18) = e
  T = sum w a takes the same errors and a's own:         |d T| / Z <= u sum p (3 a^2 + 21 a) + e sum p a
  results are rounded once, u of themselves
Alternatives and their order are the oracle's."""
import numpy as np
import pytest

from gated_deltanet_tree_amd import binding, synth
from oracle import logprobs as olp

import kv_harness as kh

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    import torch
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    binding.lib()
    return torch


class Call:
    def __init__(self, torch, logits, given=None, K=0, vocab=None, entropy=True):
        """logits: a device tensor, possibly a view."""
        N, V = logits.shape[0], vocab or logits.shape[1]
        self.N, self.V, self.K, self.given = N, V, K, given
        f32 = dict(dtype=torch.float32, device="cuda")
        self.top = (torch.full((N, K), -9, dtype=torch.int32, device="cuda"), torch.full((N, K), 9.0, **f32)) \
            if K else (None, None)
        self.given_logp = torch.full(given.shape, 9.0, **f32) if given is not None else None
        self.entropy = torch.full((N,), 9.0, **f32) if entropy else None
        need = binding.logprobs_workspace_bytes(N, V, K)
        self.ws = torch.full((need // 4 + 4,), float("nan"), **f32)
        self.args = binding.logprobs_args(logits, None if given is None else kh.dev_i32(torch, given), self.given_logp,
                                          self.top[0], self.top[1], self.entropy, self.ws, vocab=vocab)

    def run(self, stream=None):
        binding.token_logprobs(self.args, stream=stream)
        return self

    def check(self, x):
        """x [N, >= V]: the logits as float64."""
        import torch
        torch.cuda.synchronize()
        get = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
        tok, lp, giv, ent = get(self.top[0]), get(self.top[1]), get(self.given_logp), get(self.entropy)
        for r in range(self.N):
            row = x[r, :self.V]
            logp, h = olp.logprobs(row)
            clean = np.where(np.isnan(row), -np.inf, row)
            m = clean.max()
            p = np.exp(logp)
            a = np.where(p > 0, np.where(np.isfinite(clean), m - clean, 0.0), 0.0) if np.isfinite(m) else 0.0 * p
            D = float((p * a).sum())
            e = U * (3 * D + 18)

            def close(got, want):
                got, want = np.asarray(got, dtype=np.float64), np.asarray(want)
                fin = np.isfinite(want)
                assert np.array_equal(got[~fin], want[~fin]), r
                assert (got[fin] <= 0).all()
                err = np.abs(got[fin] - want[fin])
                assert (err <= e + U * np.abs(want[fin]) + 1e-38).all(), (r, (err / (e + 1e-300)).max())

            if ent is not None:
                bound = e + U * float((p * (3 * a * a + 21 * a)).sum()) + e * D + U * h + 1e-30
                assert abs(float(ent[r]) - h) <= bound, (r, ent[r], h, bound)
            if giv is not None:
                ok = (self.given[r] >= 0) & (self.given[r] < self.V)
                close(giv[r], np.where(ok, logp[np.clip(self.given[r], 0, self.V - 1)], -np.inf))
            if self.K:
                wt, wl = olp.alternatives(row, self.K)
                assert np.array_equal(tok[r], wt), (r, tok[r], wt)
                close(lp[r], wl)


def _host_rows(rng, N, V, dtype, scale=3.0):
    return kh.rng_rows(rng, (N, V), dtype, scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 7, 63, 64, 65, 255, 500, 2041, 2048, 2049, 4099, 32000, 50001])
def test_sizes(torch, V, dtype):
    rng = np.random.default_rng(V)
    x = _host_rows(rng, 3, V, dtype)
    given = rng.integers(-1, V + 1, (3, 2)).astype(np.int32)
    for K in (0, 1, 4, 64):
        Call(torch, kh.to_dev(torch, x, dtype), given, K).run().check(x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 0), (3, 5), (7, 9), (2, 64)])
def test_rows_of_any_stride_that_start_anywhere(torch, dtype, offset, pad):
    """The columns around a row hold what would win."""
    rng = np.random.default_rng(offset)
    V, N = 5003, 6
    big = np.full((N, offset + V + pad), np.inf)
    big[:, offset:offset + V] = _host_rows(rng, N, V, dtype)
    t = kh.to_dev(torch, big, dtype)[:, offset:]
    Call(torch, t, rng.integers(0, V, (N, 1)).astype(np.int32), 9, vocab=V).run().check(big[:, offset:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_logits_come_by_index(torch, dtype):
    V = 20000
    rng = np.random.default_rng(0)
    flat = np.zeros(V)
    few = rng.integers(0, 3, V).astype(np.float64)  # three values
    zeros = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    last = np.full(V, -5.0)
    last[-1] = last[-70] = 2.0
    x = np.stack([flat, few, zeros, last, flat - 1e4])
    for K in (1, 5, 64):
        Call(torch, kh.to_dev(torch, x, dtype), None, K).run().check(x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logits_that_are_not_finite(torch, dtype):
    rng = np.random.default_rng(1)
    V = 4500
    x = _host_rows(rng, 9, V, dtype)
    x[0, ::2] = -np.inf
    x[1, :] = -np.inf
    x[2, :] = np.nan
    x[3, 5:] = np.nan
    x[4, [7, 4000]] = np.inf
    x[5, :] = np.inf
    x[6, [0, 2048, V - 1]] = np.nan
    x[7, :] = -np.inf
    x[7, 4321] = -3.0
    x[8, :2048] = -np.inf
    given = np.tile(np.array([[0, 7, 4321, 4000]], dtype=np.int32), (9, 1))
    for K in (0, 6, 64):
        Call(torch, kh.to_dev(torch, x, dtype), given, K).run().check(x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extreme_logits(torch, dtype):
    """The largest finite differences, and one token that has all the weight."""
    rng = np.random.default_rng(2)
    V = 3001
    x = _host_rows(rng, 5, V, dtype)
    big = 2.0 ** 127
    x[0, ::3], x[0, 1::3] = big, -big
    x[1, 17] = 90.0
    x[2] *= 2.0 ** -130
    x[3, :] = -big
    x[3, 2000] = big
    x[4] = np.linspace(-100, 0, V)
    x = kh.host(kh.to_dev(torch, x, dtype))
    Call(torch, kh.to_dev(torch, x, dtype), None, 8).run().check(x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("order", ["rising", "falling", "turns", "runs"])
def test_the_best_may_lie_anywhere(torch, dtype, order):
    """Sorted rows, and the best ones where one thread looks for all of them."""
    V, K = 1 << 20, 64
    rng = np.random.default_rng(3)
    x = rng.standard_normal(V).astype(np.float32).astype(np.float64)
    if order == "rising":
        x = np.sort(x)
    elif order == "falling":
        x = np.sort(x)[::-1].copy()
    elif order == "turns":  # groups of 64 that are 256 apart, all of their logits
        for g in range(0, V // 64, 256):
            x[64 * g:64 * g + 64] += 10.0
    else:
        x[70000:70000 + 5000] += 10.0
    x = kh.host(kh.to_dev(torch, x[None], dtype))
    Call(torch, kh.to_dev(torch, x, dtype), None, K).run().check(x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows(torch, dtype):
    rng = np.random.default_rng(4)
    x = _host_rows(rng, 700, 3001, dtype)
    Call(torch, kh.to_dev(torch, x, dtype), rng.integers(0, 3001, (700, 1)).astype(np.int32), 5).run().check(x)


def test_large_vocabulary_without_alternatives(torch):
    rng = np.random.default_rng(5)
    x = _host_rows(rng, 1, (1 << 21) + 11, "bf16")
    Call(torch, kh.to_dev(torch, x, "bf16"), np.array([[0, 1 << 21]], dtype=np.int32)).run().check(x)


def test_outputs_may_be_left_out(torch):
    rng = np.random.default_rng(6)
    x = _host_rows(rng, 2, 300, "f32")
    t = kh.to_dev(torch, x, "f32")
    Call(torch, t, None, 0, entropy=False).run()
    Call(torch, t, None, 3, entropy=False).run().check(x)
    Call(torch, t, np.array([[1], [2]], dtype=np.int32), 0, entropy=False).run().check(x)


def test_rows_past_4_gib(torch):
    """Logits whose last rows lie beyond 2^32 bytes, by the stride alone."""
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GiB")
    V, stride = 700, 1 << 20
    buf = torch.empty((2100, stride), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(7)
    x = _host_rows(rng, 2100, V, "bf16")
    buf[:, :V] = kh.to_dev(torch, x, "bf16")
    c = Call(torch, buf, None, 3, vocab=V).run()
    torch.cuda.synchronize()
    got = c.top[0].cpu().numpy()
    for r in (0, 1, 2047, 2048, 2049, 2099):
        assert np.array_equal(got[r], olp.alternatives(x[r], 3)[0])


def test_two_calls_on_two_streams(torch):
    rng = np.random.default_rng(8)
    xs = [_host_rows(rng, 40, 30001, "bf16") for _ in range(2)]
    calls = [Call(torch, kh.to_dev(torch, x, "bf16"), None, 8) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for c, s in zip(calls, streams):
            c.run(s)
    for c, x in zip(calls, xs):
        c.check(x)


def test_captured_and_replayed(torch):
    rng = np.random.default_rng(9)
    t = torch.zeros((12, 9001), dtype=torch.float32, device="cuda")
    c = Call(torch, t, rng.integers(0, 9001, (12, 1)).astype(np.int32), 6)
    c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for _ in range(3):
        x = _host_rows(rng, 12, 9001, "f32")
        t.copy_(kh.to_dev(torch, x, "f32"))
        graph.replay()
        c.check(x)
        first = c.top[1].clone()
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(first, c.top[1])


def test_alternatives_make_a_draft_tree(torch):
    """The builder takes them as they are, and grows the tree that the oracle's scores grow."""
    from oracle import ddtree as odd
    rng = np.random.default_rng(10)
    B, L, K, V = 3, 6, 4, 1000
    x = _host_rows(rng, B * L, V, "bf16", 4.0)
    c = Call(torch, kh.to_dev(torch, x, "bf16"), None, K).run()
    c.check(x)
    lp, tok = c.top[1].cpu().numpy().reshape(B, L, K), c.top[0].cpu().numpy().reshape(B, L, K)
    for b, t in enumerate(binding.ddtree_build(lp, tok, root_tokens=[0] * B, budget=15, tau=6.0)):
        ref = odd.build(lp[b], 15, 6.0, True)
        assert t["parent"].tolist() == list(ref["parent"])
        want = [0] + [int(tok[b, d - 1, r]) for d, r in zip(t["depth"][1:], t["rank"][1:])]
        assert t["token"].tolist() == want


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [66, 129, 300, 700, 1714, 4000, 4096, 4100])
def test_as_many_alternatives_as_groups_of_64(torch, V, dtype):
    """Nearly all logits of a row are listed: drawn, rising, falling, equal, in steps, with most banned, and with the
    best ones together at one end, a few of them far above."""
    rng = np.random.default_rng(V)
    x = _host_rows(rng, 8, V, dtype)
    x[1], x[2] = np.sort(x[1]), -np.sort(x[2])
    x[3] = 1.5
    x[4] = np.round(x[4])
    x[5, rng.random(V) < 0.9] = -np.inf
    x[6, :64] = np.linspace(20, 30, 64)
    x[7, ::256] = 40.0
    x = kh.host(kh.to_dev(torch, x, dtype))  # as the kernel gets them
    for K in (1, 8, 20, 64):
        Call(torch, kh.to_dev(torch, x, dtype), None, K).run().check(x)


@pytest.mark.parametrize("V", [4032, 3900, 2500])
def test_best_logits_that_few_threads_hold(torch, V):
    """The list's keys go to 256 threads in turn: runs and steps that give a few of them most of the best ones."""
    i = np.arange(V)
    x = np.stack([i % 64, i % 256 // 4, i // 64, -i // 64, (i % 256 < 70) * 1.0, (i % 64 < 15) * (1.0 + i / V), i % 2 * 3.0])
    x = x.astype(np.float32).astype(np.float64)
    for K in (20, 63, 64):
        Call(torch, kh.to_dev(torch, x, "f32"), None, K).run().check(x)
