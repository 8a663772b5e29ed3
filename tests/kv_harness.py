"""Shared pieces of the 4-bit cache tests: caches with scattered pages and garbage in every slot
nothing was written to, the byte positions of a token by the layout's description, the oracle's
values, and error bounds.

Bounds.  Cached values and integer outputs are equal to the oracle's.  Attention, per element, with
w the oracle's softmax weights, A = sum_p w_p |V_p| and u = 2^-24:
  scores   fp32 products of exact operands: |ds| <= (d + 8) u scale sum_i |q_i K_pi| + 4 u |s|, the
           largest over the row's visible slots; exp2 and its argument add 4 u; a weight is off by
           eps_s = 2 (max ds + 4 u) relative (numerator and sum)
  sums     L fp32 terms in any order: L u relative to A
  bf16     each weight is rounded once (2^-8) for the second product, the output once (2^-8)
  fp32     the output is rounded once (u), the division adds 2 u
  |out - ref| <= (eps_s + (L + 8) u [+ 2^-8 bf16]) (A + |ref|) + (2^-8 or 3 u) |ref|
"""
from __future__ import annotations

import numpy as np

from gated_deltanet_tree_amd import binding, synth
from oracle import kv as okv

U = 2.0 ** -24


def rng_rows(rng, shape, dtype, scale=1.0):
    """fp32 draws rounded to dtype, as float64 values."""
    x = (rng.standard_normal(shape) * scale).astype(np.float32)
    return (synth.bf16_to_f32(synth.f32_to_bf16(x)) if dtype == "bf16" else x).astype(np.float64)


def to_dev(torch, x, dtype):
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def dev_i32(torch, a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def token_bytes(d, t):
    """Byte positions of slot t in a slab: key codes, key scales, value codes, value scales."""
    g, i = t // 16, t % 16
    h, qp, tt = (i // 4) % 2, i // 8, i % 4
    kc = [g * 8 * d + b * 256 + i * 16 + x for b in range(d // 32) for x in range(16)]
    ks = [g * (d // 2) + i * (d // 32) + b for b in range(d // 32)]
    vc = [g * 8 * d + (((h * 32 + m) * 2 + qp) * 4 + tt) * (d // 64) + x for m in range(32)
          for x in range(d // 64)]
    vs = [g * (d // 2) + ((h * (d // 32) + b) * 2 + qp) * 4 + tt for b in range(d // 32)]
    return kc, ks, vc, vs


class Cache:
    """A cache whose sequences hold `past` committed tokens (appended in one call) and room for
    `new` ones; every byte is garbage before (scales NaN, codes random)."""

    def __init__(self, torch, past, new, kv_heads=2, d=128, page=16, dtype="bf16", seed=0,
                 layers=1, layer=0, spare=1, missing=()):
        self.torch, self.d, self.H, self.dtype, self.page = torch, d, kv_heads, dtype, page
        self.past, self.new, self.layers, self.layer = list(past), list(new), layers, layer
        self.rng = np.random.default_rng(seed)
        S = len(past)
        need = [-(-max(p + n, 1) // page) + spare for p, n in zip(past, new)]
        n_pages, width = sum(need) + 2, max(need, default=1)
        kv = binding.alloc_kv_cache(layers, S, kv_heads, d, n_pages, page, width)
        for t in (kv.k_codes, kv.v_codes):
            t.copy_(torch.from_numpy(self.rng.integers(0, 256, t.shape, dtype=np.uint8)))
        kv.k_scales.fill_(255)
        kv.v_scales.fill_(255)
        order, at = self.rng.permutation(n_pages), 0
        table = np.full((S, width), -1, dtype=np.int32)
        for b, m in enumerate(need):
            table[b, :m] = order[at:at + m]
            at += m
        for b, i, bad in missing:  # pages that are not there
            table[b, i] = bad
        self.table = table
        kv.pages.copy_(torch.from_numpy(table))
        self.kv = kv
        # K, V: stored values of every slot of every sequence of the layer in use, past first
        self.K = [np.zeros((p + n, kv_heads, d)) for p, n in zip(past, new)]
        self.V = [np.zeros((p + n, kv_heads, d)) for p, n in zip(past, new)]
        if sum(past):
            k, v = self.rows(sum(past)), self.rows(sum(past))
            self.append(past, k, v)
            for b, o in enumerate(offsets(past)[:-1]):
                self.K[b][:past[b]], self.V[b][:past[b]] = okv.stored_pair(k[o:o + past[b]],
                                                                           v[o:o + past[b]])
        kv.length.copy_(torch.tensor(past, dtype=torch.int32))

    def rows(self, n, scale=1.0):
        return rng_rows(self.rng, (n, self.H, self.d), self.dtype, scale)

    def stack(self, x):
        """A layer's rows placed in an [layers][...] array of noise."""
        full = self.rng.standard_normal((self.layers,) + x.shape)
        full[self.layer] = x
        return to_dev(self.torch, full, self.dtype)

    def args(self, counts, **kw):
        offs = offsets(counts)
        return binding.kv_args(self.kv, offs, dev_i32(self.torch, offs), layer_begin=self.layer, **kw)

    def append(self, counts, k, v):
        binding.kv_append(self.args(counts, k=self.stack(k), v=self.stack(v)))

    def append_new(self, k=None, v=None):
        """Appends the new tokens' rows (drawn if not given)."""
        n = sum(self.new)
        k = self.rows(n) if k is None else k
        v = self.rows(n) if v is None else v
        self.append(self.new, k, v)
        for b, o in enumerate(offsets(self.new)[:-1]):
            self.K[b][self.past[b]:], self.V[b][self.past[b]:] = okv.stored_pair(
                k[o:o + self.new[b]], v[o:o + self.new[b]])
        return k, v

    def attend(self, heads, trees=None, max_length=0, q_scale=1.5, scale=None, q=None, workspace=True,
               stream=None):
        """Runs the attention; returns (q values, outputs of the layer in use)."""
        torch, T = self.torch, sum(self.new)
        q = rng_rows(self.rng, (T, heads, self.d), self.dtype, q_scale) if q is None else q
        full = np.zeros((self.layers,) + q.shape)
        full[self.layer] = q
        qd = to_dev(torch, full, self.dtype)
        out = torch.full_like(qd, float("nan"))
        kw = dict(q=qd, out=out, max_length=max_length, scale=scale)
        need = binding.attention_workspace_bytes(self.args(self.new, **kw))
        ws = torch.full((need // 4 + 4,), float("nan"), device="cuda") if workspace else None
        a = self.args(self.new, workspace=ws, **kw)
        if trees is None:
            binding.attention(a, stream=stream)
        else:
            image = binding.hld_schedule(trees)
            binding.tree_attention(a, image, torch.from_numpy(image).cuda(), stream=stream)
        torch.cuda.synchronize()
        for other in range(self.layers):
            if other != self.layer:
                assert torch.isnan(out[other].float()).all()
        return q, host(out[self.layer])

    def visible(self, b, trees=None):
        """Visibility of sequence b's new rows, pages that are not there left out."""
        see = (okv.visible_causal(self.past[b], self.new[b]) if trees is None
               else okv.visible_tree(trees[b], self.past[b]))
        pos = np.arange(see.shape[1])
        page = pos // self.page
        ids = np.where(page < self.table.shape[1], self.table[b, np.minimum(page, self.table.shape[1] - 1)], -1)
        n_pages = int(self.kv.k_codes.shape[1])
        return see & ((ids >= 0) & (ids < n_pages))[None, :]

    def check(self, q, out, trees=None, scale=None, heads=None):
        """Every output against the oracle within the derived bound; the largest share used."""
        scale = self.d ** -0.5 if scale is None else scale
        worst = 0.0
        for b, o in enumerate(offsets(self.new)[:-1]):
            n = self.new[b]
            if n == 0:
                continue
            see = self.visible(b, trees)
            worst = max(worst, check_rows(q[o:o + n], out[o:o + n], self.K[b], self.V[b], see, scale,
                                          self.dtype))
        return worst


def check_rows(q, got, K, V, see, scale, dtype, weight_half=2.0 ** -8):
    ref = okv.attention(q, K, V, see, scale)
    mag = okv.attention(q, K, np.abs(V), see, scale)
    assert np.array_equal(np.isnan(ref), np.isnan(got))
    n, Hq, d = q.shape
    G = Hq // K.shape[1]
    Kf = np.nan_to_num(np.abs(K))
    dot = np.einsum("nhgd,lhd->nhgl", np.abs(q).reshape(n, -1, G, d), Kf).reshape(n, Hq, -1)
    top = scale * np.where(see[:, None, :], dot, 0.0).max(-1, initial=0.0)
    eps = 2 * ((d + 8) * U * top + 4 * U * top + 4 * U) + (see.sum(1)[:, None] + 8) * U
    half = weight_half if dtype == "bf16" else 0.0
    out_half = 2.0 ** -8 if dtype == "bf16" else 3 * U
    bound = (eps + half)[..., None] * (mag + np.abs(ref)) + out_half * np.abs(ref) + 1e-30
    with np.errstate(invalid="ignore"):
        used = np.abs(got - ref) / bound
    used = np.nan_to_num(used)
    assert used.max(initial=0.0) <= 1.0, (used.max(), np.unravel_index(used.argmax(), used.shape))
    return float(used.max(initial=0.0))


def random_tree(rng, n, top_k=4, depth=12):
    """A parent list, parent[i] < i, in no special order."""
    parent, dep, kids = [-1], [0], [0]
    while len(parent) < n:
        p = int(rng.integers(len(parent)))
        if dep[p] < depth and kids[p] < top_k:
            kids[p] += 1
            parent.append(p)
            dep.append(dep[p] + 1)
            kids.append(0)
    return np.array(parent, dtype=np.int32)
