"""Acceptance of draft trees against the oracle: paths, lengths and next tokens are equal."""
import numpy as np
import pytest

from gated_deltanet_tree_amd import binding, synth
from oracle import accept as oaccept

import kv_harness as kh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    binding.lib()
    return torch


class Call:
    def __init__(self, torch, trees, tokens, logits, uniform, temperature, dtype="f32", stride=None,
                 shift=0, extra=2):
        """logits [T, V] fp32 values; rows start `shift` elements into a buffer of row length
        `stride`; padding holds large values."""
        self.torch, self.trees, self.tokens = torch, trees, np.asarray(tokens)
        self.image = binding.hld_schedule(trees)
        self.dev_image = torch.from_numpy(self.image).cuda()
        T, V = logits.shape
        stride = V + shift if stride is None else stride
        buf = np.full((T, stride), 99.0, dtype=np.float32)
        buf[:, shift:shift + V] = logits
        dev = kh.to_dev(torch, buf, dtype)
        self.dev_logits = dev[:, shift:shift + V]
        self.logits = kh.host(self.dev_logits)
        S = len(trees)
        width = max(len(t) for t in trees) + extra
        self.uniform = np.zeros((S, width), dtype=np.float32)
        self.uniform[:] = uniform if np.ndim(uniform) == 0 else uniform[:, :width]
        self.temperature = np.broadcast_to(np.asarray(temperature, dtype=np.float32), (S,)).copy()
        i32 = dict(dtype=torch.int32, device="cuda")
        self.path = torch.full((S, width), 55, **i32)
        self.count, self.next = torch.full((S,), 55, **i32), torch.full((S,), 55, **i32)
        self.ws = torch.full((binding.accept_workspace_bytes(self.image, V),), 255, dtype=torch.uint8,
                             device="cuda")
        self.args = binding.accept_args(
            self.image, self.dev_logits, kh.dev_i32(torch, tokens), torch.from_numpy(self.uniform).cuda(),
            torch.from_numpy(self.temperature).cuda(), self.path, self.count, self.next, self.ws)

    def run(self, stream=None):
        binding.tree_accept(self.args, self.image, self.dev_image, stream=stream)
        self.torch.cuda.synchronize()
        return self.path.cpu().numpy(), self.count.tolist(), self.next.tolist()

    def check(self):
        path, count, nxt = self.run()
        o = kh.offsets([len(t) for t in self.trees])
        for b, tree in enumerate(self.trees):
            want, tok = oaccept.accept(tree, self.tokens[o[b]:o[b + 1]], self.logits[o[b]:o[b + 1]],
                                       self.uniform[b].astype(np.float64), self.temperature[b])
            assert path[b, :count[b]].tolist() == want, b
            assert (path[b, count[b]:] == -1).all() and nxt[b] == tok, (b, nxt[b], tok)
        return count


def _draft(rng, trees, V, top=4.0):
    """Logits whose mass lies partly on the children's tokens."""
    T = sum(len(t) for t in trees)
    logits = rng.standard_normal((T, V)) * 2.0
    tokens, at = np.zeros(T, dtype=np.int32), 0
    for t in trees:
        for i, p in enumerate(t):
            if p >= 0:
                tokens[at + i] = rng.integers(V)
                logits[at + p, tokens[at + i]] = np.log(V) + top + rng.standard_normal()
        at += len(t)
    return logits.astype(np.float32), tokens


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 7, 255, 2041, 2048, 2049, 5000, 50257])
def test_trees_and_vocabularies(torch, V, dtype):
    rng = np.random.default_rng(V)
    trees = [kh.random_tree(rng, n, k, 12) for n, k in ((1, 1), (2, 1), (22, 4), (22, 4), (64, 8), (5, 1), (9, 8))]
    logits, tokens = _draft(rng, trees, V)
    u = rng.random((7, 80)).astype(np.float32)
    temp = [1.0, 0.7, 0.9, 0.0, 1.3, 0.5, 1.0]
    count = Call(torch, trees, tokens, logits, u, temp, dtype).check()
    if V > 5:
        assert max(count) > 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift,pad", [(0, 1), (1, 1), (3, 0), (7, 10), (5, 3)])
def test_rows_at_any_alignment(torch, dtype, shift, pad):
    rng = np.random.default_rng(shift)
    trees = [kh.random_tree(rng, 22, 4, 12) for _ in range(3)]
    logits, tokens = _draft(rng, trees, 4099)
    Call(torch, trees, tokens, logits, rng.random((3, 40)).astype(np.float32), 0.8, dtype,
         stride=4099 + shift + pad, shift=shift).check()


def test_largest_trees(torch):
    rng = np.random.default_rng(8)
    trees = [np.arange(-1, 1023, dtype=np.int32), np.array([-1] + [0] * 1023, dtype=np.int32),
             kh.random_tree(rng, 1000, 8, 40)]
    logits, tokens = _draft(rng, trees, 300, top=9.0)
    u = rng.random((3, 1030)).astype(np.float32) * 0.9
    count = Call(torch, trees, tokens, logits, u, 0.6).check()
    assert count[0] > 20


def test_random_numbers_at_their_ends(torch):
    rng = np.random.default_rng(11)
    trees = [kh.random_tree(rng, 22, 4, 12) for _ in range(4)]
    logits, tokens = _draft(rng, trees, 3001)
    for u in (0.0, 1.0 - 2.0 ** -24, 2.0 ** -30):
        Call(torch, trees, tokens, logits, u, 1.0).check()


def test_repeated_and_foreign_tokens(torch):
    """Siblings with one token: the first has its weight.  Tokens outside the vocabulary and the
    root's token are never matched."""
    tree = np.array([-1, 0, 0, 0, 0, 1, 1, 2], dtype=np.int32)
    V = 40
    logits = np.full((8, V), -2.0, dtype=np.float32)
    logits[:, 9] = 6.0
    for tokens in ([9, 9, 9, 3, 9, 3, 9, 9], [9, -4, V, 1 << 30, 9, 9, 9, 9], [9, 1, 2, 3, 4, 5, 6, 7],
                   [9, 9, 3, 9, 9, V, 9, 9]):
        for u in (0.01, 0.5, 0.93, 0.999):
            Call(torch, [tree], tokens, logits, u, 1.0).check()
        Call(torch, [tree], tokens, logits, 0.5, 0.0).check()


def test_masked_and_non_finite_logits(torch):
    tree = np.array([-1, 0, 0, 1, 1], dtype=np.int32)
    V = 2500
    rng = np.random.default_rng(2)
    base = rng.standard_normal((5, V)).astype(np.float32)
    tokens = [0, 17, 2400, 3, 2499]
    low = np.finfo(np.float32).min
    rows = []
    for fill in (-np.inf, low, np.nan):
        x = np.full((5, V), fill, dtype=np.float32)
        x[0, [17, 2400]] = [1.0, 1.2]
        x[1, [3, 2000]] = [0.5, 0.4]
        rows.append(x)
    every = np.full((5, V), low, dtype=np.float32)
    none = np.full((5, V), -np.inf, dtype=np.float32)
    some = base.copy()
    some[0, ::3], some[1, 17:900] = np.nan, -np.inf
    inf = base.copy()
    inf[0, [17, 5]], inf[1, 2499] = np.inf, np.inf
    for x in rows + [every, none, some, inf]:
        for u in (0.02, 0.4, 0.7, 0.99):
            for T in (1.0, 0.0, 1e-30, 1e30, float("nan"), float("inf"), -1.0):
                Call(torch, [tree], tokens, x, u, T).check()


def test_greedy_takes_the_lowest_of_equal_logits(torch):
    tree = np.array([-1, 0, 1], dtype=np.int32)
    for where in ([5, 3000], [2047, 2048], [0, 4999], [4998, 4999]):
        x = np.zeros((3, 5000), dtype=np.float32)
        x[:, where] = 1.0
        assert Call(torch, [tree], [0, where[0], 1], x, 0.5, 0.0, "bf16").check() == [2]
        assert Call(torch, [tree], [0, where[1], 1], x, 0.5, 0.0, "bf16").check() == [1]


def test_first_token_has_the_targets_frequencies(torch):
    """2000 sequences with evenly spaced random numbers: every token's count is its probability
    times 2000, to within one."""
    S, V = 2000, 11
    rng = np.random.default_rng(6)
    row = rng.standard_normal(V).astype(np.float32)
    tree = np.array([-1, 0, 0], dtype=np.int32)
    logits = np.tile(row, (3 * S, 1))
    tokens = np.tile([0, 4, 7], S).astype(np.int32)
    u = np.repeat(((np.arange(S) + 0.5) / S)[:, None], 8, axis=1).astype(np.float32)
    c = Call(torch, [tree] * S, tokens, logits, u, 0.9)
    path, count, nxt = c.run()
    drawn = np.array([[0, 4, 7][path[b, 1]] if count[b] > 1 else nxt[b] for b in range(S)])
    p = np.exp(row.astype(np.float64) / np.float64(np.float32(0.9)))
    assert np.abs(np.bincount(drawn, minlength=V) - S * p / p.sum()).max() <= 1.0


def test_streams_graphs_and_repeats(torch):
    rng = np.random.default_rng(12)
    trees = [kh.random_tree(rng, 22, 4, 12) for _ in range(5)]
    logits, tokens = _draft(rng, trees, 9000)
    c = Call(torch, trees, tokens, logits, rng.random((5, 40)).astype(np.float32), 0.9)
    c.check()
    first = [t.clone() for t in (c.path, c.count, c.next)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for t in (c.path, c.count, c.next):
        t.fill_(77)
    torch.cuda.synchronize()
    c.run(stream=s)
    assert all(torch.equal(a, b) for a, b in zip(first, (c.path, c.count, c.next)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.tree_accept(c.args, c.image, c.dev_image)
    for step in range(4):
        logits, _ = _draft(rng, trees, 9000)
        c.dev_logits.copy_(kh.to_dev(torch, logits, "f32"))
        for t in (c.path, c.count, c.next):
            t.fill_(77)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (c.path, c.count, c.next)]
        c.logits = kh.host(c.dev_logits)
        c.check()  # eager, on the same inputs
        assert all(torch.equal(a, b) for a, b in zip(got, (c.path, c.count, c.next)))


def test_batched_workload_trees(torch):
    trees = [synth.workload_tree("batched", b) for b in range(32)]
    rng = np.random.default_rng(13)
    logits, tokens = _draft(rng, trees, 32000)
    temp = np.where(np.arange(32) % 4 == 3, 0.0, 0.8)
    count = Call(torch, trees, tokens, logits, rng.random((32, 40)).astype(np.float32), temp, "bf16").check()
    assert np.mean(count) > 2


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_last_child_takes_the_end_where_only_children_have_weight(torch, dtype):
    """u = 1 - 2^-24 over nodes whose weight is all their children's: the last child with weight is
    accepted, whichever way the sum of the weights rounds."""
    S, V = 1500, 70
    rng = np.random.default_rng(31)
    trees = [np.array([-1, 0, 0, 0, 2], dtype=np.int32)] * S
    logits = np.full((5 * S, V), -np.inf, dtype=np.float32)
    tokens = np.zeros(5 * S, dtype=np.int32)
    for b in range(S):
        kids = rng.choice(V, 3, replace=False)
        tokens[5 * b + 1:5 * b + 4] = kids
        tokens[5 * b + 4] = 3
        logits[5 * b, kids] = rng.standard_normal(3) * 2.0
        logits[5 * b + 1:5 * b + 5] = rng.standard_normal((4, V))
    c = Call(torch, trees, tokens, logits, 1.0 - 2.0 ** -24, 0.9, dtype)
    assert set(c.check()) == {2}
    assert (c.path.cpu().numpy()[:, 1] == 3).all()


@pytest.mark.parametrize("V,S", [(300, 400), (2049, 300), (60001, 24)])
def test_random_numbers_next_to_a_border(torch, V, S):
    """u the fp32 numbers on either side of a child's border, as 64 bits place it."""
    rng = np.random.default_rng(V)
    tree = np.array([-1, 0, 0, 0, 1, 2], dtype=np.int32)
    n = len(tree)
    logits, tokens = _draft(rng, [tree] * S, V, top=1.0)
    temp = np.where(np.arange(S) % 2, 0.8, 1.1).astype(np.float32)
    u = np.full((S, 8), 0.4, dtype=np.float32)
    for b in range(S):
        w = oaccept.weights(logits[n * b], temp[b])
        kids = [t for _, t in oaccept.child_tokens(tree, tokens[n * b:n * b + n], 0, V)]
        border = np.float32(w[kids[:1 + b % len(kids)]].sum() / w.sum())
        u[b, 0] = (np.nextafter(border, np.float32(0)), border, np.nextafter(border, np.float32(1)))[b // 2 % 3]
    Call(torch, [tree] * S, tokens, logits, u, temp).check()
