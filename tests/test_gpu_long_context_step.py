"""Speculative steps over a long context as a serving loop runs them, in a cache whose pages are handed
out on the device: draft logits -> alternatives -> tree -> pages and slots -> append, page selection and
sparse tree attention per attention layer -> acceptance -> commit -> bounds of the filled pages -> what the
rejected nodes had reserved goes back.  Every piece is checked against the oracles."""
import numpy as np
import pytest

from gated_deltanet_tree_amd import binding, synth
from oracle import accept as oaccept
from oracle import kv as okv
from oracle import logprobs as olp
from oracle import pages as op
from oracle import sparse as osp

import kv_harness as kh

pytestmark = pytest.mark.gpu

S, HKV, GROUP, D, VOCAB, LAYERS, PAGE, TOP = 3, 2, 3, 64, 900, 2, 16, 4
POSITIONS, TOPK, BUDGET, N_PAGES, WIDTH = 5, 4, 14, 60, 16


def test_steps_over_a_long_context():
    import torch
    binding.lib()
    rng = np.random.default_rng(31)
    i32 = dict(dtype=torch.int32, device="cuda")
    kv = binding.alloc_kv_cache(LAYERS, S, HKV, D, N_PAGES, PAGE, WIDTH)
    refs = binding.alloc_kv_refs(kv)
    bounds = binding.alloc_kv_bounds(kv)
    table, count, length = [[-1] * WIDTH for _ in range(S)], [0] * N_PAGES, [0] * S
    hist = [[[np.zeros((0, HKV, D))] * 2 for _ in range(S)] for _ in range(LAYERS)]

    def reserve(new, offs, dev_offs, depth=None):
        T = int(offs[-1])
        out = dict(missing=torch.full((S,), -1, **i32), positions=torch.full((T,), -1, **i32),
                   slots=torch.full((T,), -7, dtype=torch.int64, device="cuda"))
        a = (kv.pages, kv.length, refs, PAGE, offs, dev_offs)
        dep = None if depth is None else kh.dev_i32(torch, depth)
        ws = torch.empty(binding.pages_workspace_bytes(binding.pages_args(*a)), dtype=torch.uint8, device="cuda")
        args = binding.pages_args(*a, depth=dep, workspace=ws, **out)
        binding.kv_reserve(args)
        missing, slots, positions = op.reserve(table, count, length, new, PAGE, depth)
        assert out["missing"].tolist() == missing == [0] * S
        assert out["slots"].tolist() == slots and out["positions"].tolist() == positions
        return args

    def kept(args, keep):
        binding.kv_release(args, kv.length)
        op.release(table, count, keep, PAGE)
        assert kv.pages.cpu().numpy().tolist() == table and refs.cpu().numpy().tolist() == count

    # prompts
    prompt = [150, 33, 0]
    offs = kh.offsets(prompt)
    dev = kh.dev_i32(torch, offs)
    pages = reserve(prompt, offs, dev)
    k, v = (kh.rng_rows(rng, (LAYERS, sum(prompt), HKV, D), "bf16") for _ in range(2))
    a = binding.kv_args(kv, offs, dev, k=kh.to_dev(torch, k, "bf16"), v=kh.to_dev(torch, v, "bf16"), n_layers=LAYERS)
    binding.kv_append(a)
    binding.kv_commit(a, None, kh.dev_i32(torch, prompt), kv.length)
    binding.kv_bounds(a, binding.sparse_args(a, bounds))
    for l in range(LAYERS):
        for b in range(S):
            hist[l][b] = list(okv.stored_pair(k[l, offs[b]:offs[b + 1]], v[l, offs[b]:offs[b + 1]]))
    length = list(prompt)
    kept(pages, length)

    for step in range(4):
        # drafts: alternatives of the draft's logits make the trees
        draft = kh.rng_rows(rng, (S * POSITIONS, VOCAB), "bf16", 3.0)
        f32 = dict(dtype=torch.float32, device="cuda")
        tok, lp = torch.empty((S * POSITIONS, TOPK), **i32), torch.empty((S * POSITIONS, TOPK), **f32)
        ws = torch.empty(binding.logprobs_workspace_bytes(S * POSITIONS, VOCAB, TOPK), dtype=torch.uint8, device="cuda")
        binding.token_logprobs(binding.logprobs_args(kh.to_dev(torch, draft, "bf16"), top_token=tok, top_logp=lp,
                                                     workspace=ws))
        for r in range(S * POSITIONS):
            assert tok[r].tolist() == olp.alternatives(draft[r], TOPK)[0].tolist()
        built = binding.ddtree_build(lp.cpu().numpy().reshape(S, POSITIONS, TOPK),
                                     tok.cpu().numpy().reshape(S, POSITIONS, TOPK), root_tokens=[1, 2, 3],
                                     budget=BUDGET, tau=float("inf"))
        trees, tokens = [t["parent"] for t in built], np.concatenate([t["token"] for t in built])
        image = binding.hld_schedule(trees)
        dev_image = torch.from_numpy(image).cuda()
        new = [len(t) for t in trees]
        offs, T = kh.offsets(new), sum(new)
        dev = dev_image[16:16 + S + 1]
        pages = reserve(new, offs, dev, binding.schedule_view(image)["node_depth"].tolist())
        # attention layers
        k, v = (kh.rng_rows(rng, (LAYERS, T, HKV, D), "bf16") for _ in range(2))
        q = kh.rng_rows(rng, (LAYERS, T, HKV * GROUP, D), "bf16", 1.5)
        kd, vd, qd = (kh.to_dev(torch, x, "bf16") for x in (k, v, q))
        out = torch.zeros_like(qd)
        sel = torch.full((LAYERS, T, HKV, TOP), -1, **i32)
        for l in range(LAYERS):
            kw = dict(q=qd, out=out, k=kd, v=vd, layer_begin=l)

            def sparse(x):
                return binding.sparse_args(x, bounds, sel, TOP, share_tokens=0, keep_first=1, keep_last=1)

            a = binding.kv_args(kv, offs, dev, **kw)
            ws = torch.empty(binding.sparse_workspace_bytes(a, sparse(a)) + 16, dtype=torch.uint8, device="cuda")
            a = binding.kv_args(kv, offs, dev, workspace=ws, **kw)
            binding.kv_append(a)
            binding.kv_select(a, sparse(a))
            binding.sparse_tree_attention(a, sparse(a), image, dev_image)
        # acceptance and commit
        logits = kh.rng_rows(rng, (T, VOCAB), "bf16", 2.0)
        for b, t in enumerate(trees):
            for i, p in enumerate(t):
                if p >= 0:
                    logits[offs[b] + p, tokens[offs[b] + i]] += 9.0
        logits = synth.bf16_to_f32(synth.f32_to_bf16(logits.astype(np.float32))).astype(np.float64)
        u, temp = rng.random((S, BUDGET)).astype(np.float32), np.array([1.0, 0.0, 0.8], dtype=np.float32)
        path, taken, nxt = torch.empty((S, BUDGET), **i32), torch.empty(S, **i32), torch.empty(S, **i32)
        ws = torch.empty(binding.accept_workspace_bytes(image, VOCAB), dtype=torch.uint8, device="cuda")
        binding.tree_accept(
            binding.accept_args(image, kh.to_dev(torch, logits, "bf16"), kh.dev_i32(torch, tokens),
                                torch.from_numpy(u).cuda(), torch.from_numpy(temp).cuda(), path, taken, nxt, ws),
            image, dev_image)
        a = binding.kv_args(kv, offs, dev, k=kd, v=vd, n_layers=LAYERS)
        binding.kv_commit(a, path, taken, kv.length)
        binding.kv_bounds(a, binding.sparse_args(a, bounds))
        torch.cuda.synchronize()
        # ---- against the oracles ----
        chosen, got_bounds = sel.cpu().numpy(), kh.host(bounds)
        for b, tree in enumerate(trees):
            sl = slice(offs[b], offs[b + 1])
            want, token = oaccept.accept(tree, tokens[sl], logits[sl], u[b].astype(np.float64), temp[b])
            assert path[b, :int(taken[b])].tolist() == want and int(nxt[b]) == token
            full = length[b] // PAGE
            see = okv.visible_tree(tree, length[b])
            for l in range(LAYERS):
                ks, vs = okv.stored_pair(k[l, sl], v[l, sl])
                K, V = np.concatenate([hist[l][b][0], ks]), np.concatenate([hist[l][b][1], vs])
                entries = osp.select(q[l, sl], K, PAGE, full, TOP, 0, 1, 1)[0]
                assert np.array_equal(chosen[l, offs[b], :, :min(TOP, full)], entries)
                for h in range(HKV):
                    cols = slice(h * GROUP, (h + 1) * GROUP)
                    kh.check_rows(q[l, sl][:, cols], kh.host(out[l, sl])[:, cols], K[:, h:h + 1], V[:, h:h + 1],
                                  osp.visible(see, entries[h], PAGE, full), D ** -0.5, "bf16")
                hist[l][b] = [np.concatenate([hist[l][b][0], ks[want]]), np.concatenate([hist[l][b][1], vs[want]])]
            length[b] += len(want)
            for l in range(LAYERS):
                for i in range(length[b] // PAGE):
                    for h in range(HKV):
                        assert np.array_equal(got_bounds[l, table[b][i], h],
                                              osp.limits(hist[l][b][0][i * PAGE:(i + 1) * PAGE, h]))
        assert kv.length.tolist() == length
        kept(pages, length)
    assert length[0] // PAGE > TOP and sum(length) > sum(prompt) + 4 * S
