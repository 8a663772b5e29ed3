"""Sparse attention over a kv_harness cache: bounds, selections and outputs against the oracle.
Bounds are equal to the oracle's, selections too (scores are fp64 sums, the draws have no two pages
nearer than their rounding unless they are equal), outputs within kv_harness's bound over the slots
that the oracle's selection leaves."""
from __future__ import annotations

import numpy as np

from gated_deltanet_tree_amd import binding
from oracle import kv as okv
from oracle import sparse as osp

import kv_harness as kh


class SparseCache(kh.Cache):
    def build_bounds(self):
        """Bounds of every full page of the committed tokens; all others keep a mark."""
        torch = self.torch
        self.bounds = binding.alloc_kv_bounds(self.kv)
        self.bounds.fill_(77.0)
        a = self.args(self.past)
        binding.kv_bounds(a, binding.sparse_args(a, self.bounds))
        torch.cuda.synchronize()
        return self.bounds

    def there(self, b):
        full = self.past[b] // self.page
        ids = self.table[b, :full]
        return (ids >= 0) & (ids < int(self.kv.k_codes.shape[1]))

    def check_bounds(self):
        got = kh.host(self.bounds)
        want = np.full(got.shape, 77.0)
        for b, p in enumerate(self.past):
            for i in np.flatnonzero(self.there(b)):
                for h in range(self.H):
                    hi, lo = osp.limits(self.K[b][i * self.page:(i + 1) * self.page, h])
                    # a NaN key marks 32 channels at least, and the score is NaN either way
                    want[self.layer, self.table[b, i], h] = [hi, lo]
        bad = np.isnan(want)
        assert np.isnan(got[bad]).all() and np.array_equal(got[~bad], want[~bad])

    def select_and_attend(self, heads, top, share=1, first=0, last=0, trees=None, max_length=0, q=None, q_scale=1.5,
                          selected=None, stream=None, scale=None):
        """Returns (q values, selections [T][Hkv][top], outputs) of the layer in use."""
        torch, T = self.torch, sum(self.new)
        q = kh.rng_rows(self.rng, (T, heads, self.d), self.dtype, q_scale) if q is None else q
        full = np.zeros((self.layers,) + q.shape)
        full[self.layer] = q
        qd = kh.to_dev(torch, full, self.dtype)
        out = torch.full_like(qd, float("nan"))
        given = selected is not None
        sel = torch.full((self.layers, T, self.H, top), -7, dtype=torch.int32, device="cuda")
        if given:
            sel[self.layer] = kh.dev_i32(torch, selected)
        kw = dict(q=qd, out=out, max_length=max_length, scale=scale)

        def sparse(a):
            return binding.sparse_args(a, self.bounds, sel, top, share, first, last)

        a = self.args(self.new, **kw)
        need = binding.sparse_workspace_bytes(a, sparse(a))
        ws = torch.full((need // 4 + 4,), float("nan"), device="cuda")
        a = self.args(self.new, workspace=ws, **kw)
        x = sparse(a)
        if not given:
            binding.kv_select(a, x, stream=stream)
        if trees is None:
            binding.sparse_attention(a, x, stream=stream)
        else:
            image = binding.hld_schedule(trees)
            binding.sparse_tree_attention(a, x, image, torch.from_numpy(image).cuda(), stream=stream)
        torch.cuda.synchronize()
        for other in range(self.layers):
            if other != self.layer:
                assert torch.isnan(out[other].float()).all() and (given or (sel[other] == -7).all())
        return q, sel[self.layer].cpu().numpy(), kh.host(out[self.layer])

    def oracle_selections(self, b, q, top, share, first, last):
        return osp.select(q, self.K[b], self.page, self.past[b] // self.page, top, share, first, last, self.there(b))

    def check_sparse(self, q, sel, out, top, share=1, first=0, last=0, trees=None, chosen=None, scale=None):
        """chosen: selections [T][Hkv][top] given to the attention, instead of the oracle's."""
        scale = self.d ** -0.5 if scale is None else scale
        for b, o in enumerate(kh.offsets(self.new)[:-1]):
            n, full = self.new[b], self.past[b] // self.page
            if n == 0:
                continue
            G = q.shape[1] // self.H
            see = self.visible(b, trees)
            if chosen is None:
                want = self.oracle_selections(b, q[o:o + n], top, share, first, last)
            for g, (i0, i1) in enumerate(osp.selections(n, share)):
                if chosen is None:
                    k = min(top, full)
                    assert np.array_equal(sel[o + i0, :, :k], want[g]), (b, g)
                    assert (sel[o + i0, :, k:] == -1).all()
                    assert (sel[o + i0 + 1:o + i1] == -7).all()
                for h in range(self.H):
                    use = want[g][h] if chosen is None else [
                        e for e in chosen[o + i0, h, :min(top, full)] if 0 <= e < full]
                    part = osp.visible(see[i0:i1], use, self.page, full)
                    kh.check_rows(q[o + i0:o + i1, h * G:(h + 1) * G], out[o + i0:o + i1, h * G:(h + 1) * G],
                                  self.K[b][:, h:h + 1], self.V[b][:, h:h + 1], part, scale, self.dtype)
