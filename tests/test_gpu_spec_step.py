"""Speculative steps of a small hybrid stack as a serving loop runs them: drafts -> tree -> cache
append and tree attention per attention layer, recurrent verify per recurrent layer -> acceptance
-> commit of both.  Every piece is checked against the oracles, and the caches after two steps hold
what a plain token-by-token run would have put there."""
import numpy as np
import pytest

from gated_deltanet_tree_amd import binding, synth
from oracle import accept as oaccept
from oracle import gdn as ogdn
from oracle import kv as okv

import gpu_harness as gh
import kv_harness as kh

pytestmark = pytest.mark.gpu

S, HKV, GROUP, D, VOCAB, LAYERS, PAGE = 3, 2, 3, 128, 700, 2, 16


def test_two_steps_of_a_hybrid_stack():
    import torch
    rng = np.random.default_rng(21)
    kv = binding.alloc_kv_cache(LAYERS, S, HKV, D, 30, PAGE, 8)
    kv.pages.copy_(torch.from_numpy(rng.permutation(30)[:24].reshape(3, 8).astype(np.int32)))
    # prompts fill the attention caches and are committed without moving rows
    prompt = [5, 0, 33]
    offs = kh.offsets(prompt)
    hist_k = [[np.zeros((0, HKV, D))] * S for _ in range(LAYERS)]
    hist_v = [[np.zeros((0, HKV, D))] * S for _ in range(LAYERS)]
    k, v = (kh.rng_rows(rng, (LAYERS, sum(prompt), HKV, D), "bf16") for _ in range(2))
    a = binding.kv_args(kv, offs, kh.dev_i32(torch, offs), k=kh.to_dev(torch, k, "bf16"),
                        v=kh.to_dev(torch, v, "bf16"), n_layers=LAYERS)
    binding.kv_append(a)
    binding.kv_commit(a, None, kh.dev_i32(torch, prompt), kv.length)
    for l in range(LAYERS):
        for b in range(S):
            hist_k[l][b], hist_v[l][b] = okv.stored_pair(k[l, offs[b]:offs[b + 1]], v[l, offs[b]:offs[b + 1]])
    H, Cch = 2, 0
    state0 = np.stack([synth.initial_state(7, 0, b, H, D) for b in range(S)])
    gdn_state = [state0[b].astype(np.float64) for b in range(S)]
    layers = None
    length = list(prompt)
    for step in range(2):
        drafts = [synth.draft_scores(40 + step, step, b, 8, 4) for b in range(S)]
        built = binding.ddtree_build(np.stack([d[0] for d in drafts]), np.stack([d[1] for d in drafts]),
                                     root_tokens=[1, 2, 3], budget=18, tau=float("inf"))
        trees = [t["parent"] for t in built]
        tokens = np.concatenate([t["token"] for t in built])
        batch = gh.Batch(trees, 1, H, D, Cch, max_nodes=18, mode="ut")
        if layers is None:
            batch.set_state(state0[None])
            layers = batch.layers
        else:
            batch.layers = layers
        T, toffs = batch.T, batch.offs
        # attention layers
        k, v = (kh.rng_rows(rng, (LAYERS, T, HKV, D), "bf16") for _ in range(2))
        q = kh.rng_rows(rng, (LAYERS, T, HKV * GROUP, D), "bf16", 1.5)
        kd, vd, qd = (kh.to_dev(torch, x, "bf16") for x in (k, v, q))
        out = torch.zeros_like(qd)
        dev_offs = batch.dev_image[16:16 + S + 1]
        kw = dict(q=qd, out=out, k=kd, v=vd)
        for l in range(LAYERS):
            need = binding.attention_workspace_bytes(
                binding.kv_args(kv, toffs, dev_offs, layer_begin=l, **kw))
            ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
            al = binding.kv_args(kv, toffs, dev_offs, workspace=ws, layer_begin=l, **kw)
            binding.kv_append(al)
            binding.tree_attention(al, batch.image, batch.dev_image)
        # a recurrent layer
        h = gh.tiny_inputs(trees, step, H, D, 4, "bf16", 7)
        h.pop("x")
        from gated_deltanet_tree_amd import workload
        inp = workload.StepInputs(**{n: workload._to_torch(x, "bf16", "cuda") for n, x in h.items()}, x=None)
        binding.tree_verify_ut(batch.vargs(inp, 0), batch.image, batch.dev_image)
        # logits, acceptance, both commits
        logits = kh.rng_rows(rng, (T, VOCAB), "bf16", 2.0)
        for b, t in enumerate(trees):
            for i, p in enumerate(t):
                if p >= 0:
                    logits[toffs[b] + p, tokens[toffs[b] + i]] += 9.0
        logits = synth.bf16_to_f32(synth.f32_to_bf16(logits.astype(np.float32))).astype(np.float64)
        u = rng.random((S, 18)).astype(np.float32)
        temp = np.array([1.0, 0.0, 0.8], dtype=np.float32)
        i32 = dict(dtype=torch.int32, device="cuda")
        path, count, nxt = torch.empty((S, 18), **i32), torch.empty(S, **i32), torch.empty(S, **i32)
        ws2 = torch.empty(binding.accept_workspace_bytes(batch.image, VOCAB), dtype=torch.uint8, device="cuda")
        binding.tree_accept(
            binding.accept_args(batch.image, kh.to_dev(torch, logits, "bf16"), kh.dev_i32(torch, tokens),
                                torch.from_numpy(u).cuda(), torch.from_numpy(temp).cuda(), path, count, nxt, ws2),
            batch.image, batch.dev_image)
        binding.kv_commit(binding.kv_args(kv, toffs, dev_offs, k=kd, v=vd, n_layers=LAYERS), path, count, kv.length)
        paths = [path[b, :int(count[b])].cpu().numpy() for b in range(S)]
        batch.commit(inp, paths)
        torch.cuda.synchronize()
        # ---- against the oracles ----
        h64 = gh.widen_inputs(h, "bf16")
        for b, tree in enumerate(trees):
            sl = slice(toffs[b], toffs[b + 1])
            want, tok = oaccept.accept(tree, tokens[sl], logits[sl], u[b].astype(np.float64), temp[b])
            assert paths[b].tolist() == want and int(nxt[b]) == tok
            see = okv.visible_tree(tree, length[b])
            for l in range(LAYERS):
                ks, vs = okv.stored_pair(k[l, sl], v[l, sl])
                kh.check_rows(q[l, sl], kh.host(out[l, sl]), np.concatenate([hist_k[l][b], ks]),
                              np.concatenate([hist_v[l][b], vs]), see, D ** -0.5, "bf16")
                hist_k[l][b] = np.concatenate([hist_k[l][b], ks[want]])
                hist_v[l][b] = np.concatenate([hist_v[l][b], vs[want]])
            seq = {n: x[0, sl] for n, x in h64.items()}
            r = gh.oracle_pair(tree, gdn_state[b], None, None, seq, "ut", H, D)
            gh.assert_outputs(gh.to_np(batch.out[0])[sl], r["o"], what="recurrent layer")
            gdn_state[b] = ogdn.replay(gdn_state[b], seq["k"], seq["v"], seq["beta"], seq["gate"], want)
            length[b] += len(want)
        assert kv.length.tolist() == length
    assert sum(length) > sum(prompt) + 2 * S  # drafts were accepted
    # what the caches hold is what token-by-token appends would have left
    offs = kh.offsets(length)
    ko = torch.empty((LAYERS, int(offs[-1]), HKV, D), dtype=torch.bfloat16, device="cuda")
    vo = torch.empty_like(ko)
    binding.kv_read(binding.kv_args(kv, offs, kh.dev_i32(torch, offs), k=ko, v=vo, n_layers=LAYERS),
                    begin=torch.zeros(S, **i32))
    for l in range(LAYERS):
        assert np.array_equal(kh.host(ko[l]), np.concatenate(hist_k[l]))
        assert np.array_equal(kh.host(vo[l]), np.concatenate(hist_v[l]))
