"""Cases, inputs and plain forms of what a speculative step needs before and beside its attention:
log probabilities of rows of logits (given tokens, entropy, sorted alternatives for the draft-tree
builder), the page tables and slot maps of the paged key/value cache, and sparse attention over the
pages of the 4-bit cache that a cheap score selects for each query.

Alternatives are sorted by value, equal ones by index.  Tables without a page for a slot take the
lowest free ids in order of sequence and entry.  A page's score for a query is the largest q.k that
its channelwise bounds allow, max over the rows that share a selection; the pages that are full at the
committed length compete, all later slots are always seen.

The 4-bit cache: 32 consecutive channels of one (token, kv head) share a power of two 2^e, held as the
byte e + 127; elements are the 4-bit floats {0, .5, 1, 1.5, 2, 3, 4, 6} with a sign.  A page holds, per
kv head, groups of 16 tokens:
    key codes    [group][block of 32 channels][token][16 bytes], channel 2i in byte i's low half
    key scales   [group][token][block]
    value codes  [group][h][m][qp][t][d/64 bytes] with token 8 qp + 4 h + t and channel
                 (d/32) m + k in half byte k of the piece (low half first)
    value scales [group][h][block][qp][t]
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------

def listed():
    return [
        # one user's draft: the candidates of 12 positions for the tree builder
        dict(name="draft_one", op="logprobs", rows=12, vocab=32000, pad=0, dtype="f32", topk=4, given=0, banned=0),
        # the batched workload's 32 drafts of 12 positions over a large vocabulary
        dict(name="draft_batched", op="logprobs", rows=384, vocab=131072, pad=64, dtype="bf16", topk=4, given=0,
             banned=0),
        # scoring of a prompt: the token that came, and 20 alternatives, under a list of banned tokens
        dict(name="prompt_scores", op="logprobs", rows=2047, vocab=32001, pad=0, dtype="f32", topk=20, given=1,
             banned=100),
        # the batched workload's trees get their slots in a pool of medium size
        dict(name="pages_batched", op="pages", seqs=32, new_lo=22, new_hi=22, past_lo=2000, past_hi=16000, page=64,
             spare=1000, tree=True, shape=1),
        # admission of many prompts into a large pool of small pages
        dict(name="pages_prompts", op="pages", seqs=256, new_lo=500, new_hi=4096, past_lo=0, past_hi=30000, page=16,
             spare=40000, tree=False, shape=2),
        # after a step of the batched workload: the pages that its commit completed, in 16 layers
        dict(name="bounds_step", op="bounds", seqs=32, new_lo=22, new_hi=22, past_lo=2000, past_hi=4000, kv_heads=8,
             dim=128, page=64, layers=16, dtype="bf16", shape=3),
        # after long prompts, one layer
        dict(name="bounds_prompt", op="bounds", seqs=4, new_lo=20000, new_hi=40000, past_lo=0, past_hi=100,
             kv_heads=8, dim=128, page=64, layers=1, dtype="bf16", shape=4),
        # the smallest call: one token of one conversation
        dict(name="sparse_one", op="sparse", seqs=1, new_lo=1, new_hi=1, past_lo=20011, past_hi=20011, heads=16,
             kv_heads=4, dim=64, page=32, top=32, share=1, first=1, last=1, dtype="bf16", shape=5),
        # plain decode of a batch with long caches
        dict(name="sparse_batched", op="sparse", seqs=32, new_lo=1, new_hi=1, past_lo=8000, past_hi=40000, heads=32,
             kv_heads=8, dim=128, page=64, top=32, share=1, first=1, last=2, dtype="bf16", shape=6),
        # draft trees on long contexts: a tree's nodes share their pages
        dict(name="sparse_trees", op="tree", seqs=8, new_lo=22, new_hi=22, topk=4, depth=12, past_lo=16000,
             past_hi=65000, heads=48, kv_heads=8, dim=128, page=64, top=64, share=0, first=1, last=2, dtype="bf16",
             shape=7),
        # chunks of prompts, 16 tokens to a selection
        dict(name="sparse_chunks", op="sparse", seqs=4, new_lo=200, new_hi=512, past_lo=8000, past_hi=20000, heads=32,
             kv_heads=8, dim=128, page=64, top=32, share=16, first=1, last=2, dtype="bf16", shape=8),
        # two very long contexts with wide heads, kept in 32 bits
        dict(name="sparse_long_f32", op="sparse", seqs=2, new_lo=1, new_hi=2, past_lo=200003, past_hi=262000,
             heads=16, kv_heads=2, dim=256, page=128, top=64, share=1, first=1, last=2, dtype="f32", shape=9),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    cap = [work(c) for c in listed()]
    cap_bytes, cap_flops = max(w["bytes"] for w in cap), max(w["flops"] for w in cap)
    while True:
        op = rng.choice(["logprobs", "logprobs", "pages", "bounds", "sparse", "sparse", "tree"])
        c = dict(op=op)
        if op == "logprobs":
            vocab = _log_int(rng, 101, 160001)
            c.update(rows=_log_int(rng, 1, 2048), vocab=vocab, pad=rng.choice([0, 0, 8, 63]),
                     dtype=rng.choice(["bf16", "f32"]), topk=min(rng.choice([0, 1, 4, 8, 16, 20, 64]), vocab // 4),
                     given=rng.choice([0, 1, 1, 3]), banned=rng.choice([0, 0, 30]))
        else:
            seqs = _log_int(rng, 1, 48)
            c.update(seqs=seqs, shape=rng.randrange(1 << 30), page=rng.choice([16, 32, 64, 128, 256]))
            past = _log_int(rng, 1, 65536)
            n = _log_int(rng, 1, 4096 if op in ("pages", "bounds") else 64 if op == "tree" else 300)
            c.update(new_lo=max(1, n // 3), new_hi=n, past_lo=rng.randint(0, past), past_hi=past)
            if op == "pages":
                c.update(seqs=_log_int(rng, 1, 300), spare=_log_int(rng, 1, 20000), tree=rng.random() < 0.3)
                if c["tree"]:
                    c["new_hi"] = min(c["new_hi"], 64)
                    c["new_lo"] = min(c["new_lo"], c["new_hi"])
            else:
                kvh = rng.choice([1, 2, 3, 4, 8])
                c.update(kv_heads=kvh, dim=rng.choice([64, 128, 256]), dtype=rng.choice(["bf16", "bf16", "f32"]))
            if op == "bounds":
                c["layers"] = _log_int(rng, 1, 16)
            elif op in ("sparse", "tree"):
                top = _log_int(rng, 1, 128)
                first = rng.randint(0, min(2, top))
                c.update(heads=kvh * rng.choice([1, 2, 3, 4, 6, 8, 16]), top=top, first=first,
                         last=rng.randint(0, min(2, top - first)))
                if op == "tree":
                    c.update(share=0, topk=rng.randint(2, 8) + n // 8, depth=rng.randint(6, 16))
                else:
                    c["share"] = rng.choice([0, 1, 1, 2, 8, 16, 64])
                    if c["share"] and seqs * n / c["share"] > 300:
                        continue
        w = work(c)
        if w["bytes"] <= cap_bytes and w["flops"] <= cap_flops:
            return c


def _tree(rng, n, topk, depth):
    """A parent list grown from a main chain, parent[i] < i (children in no special order)."""
    main = min(n, depth + 1)
    parent, dep, kids = list(range(-1, main - 1)), list(range(main)), [1] * (main - 1) + [0]
    while len(parent) < n:
        p = rng.randrange(len(parent))
        if dep[p] < depth and kids[p] < topk:
            kids[p] += 1
            parent.append(p)
            dep.append(dep[p] + 1)
            kids.append(0)
    return parent


def _shapes(case):
    """Ragged sizes of a case: new tokens and cached tokens of every sequence, and its trees."""
    rng = random.Random(case["shape"])
    S = case["seqs"]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(S)]
    past = [rng.randint(case["past_lo"], case["past_hi"]) for _ in range(S)]
    out = dict(new=new, past=past)
    if case["op"] == "tree":
        out["trees"] = [_tree(rng, n, case["topk"], case["depth"]) for n in new]
    elif case["op"] == "pages" and case["tree"]:
        out["trees"] = [_tree(rng, n, 12, 12) for n in new]
    return out


def _depths(tree):
    d = []
    for p in tree:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _groups(n, share):
    """[first, last) tokens of the groups that share a selection."""
    share = share or max(n, 1)
    return [(i, min(n, i + share)) for i in range(0, n, share)]


def work(case):
    if case["op"] == "logprobs":
        size = 2 if case["dtype"] == "bf16" else 4
        n = case["rows"] * case["vocab"]
        return dict(bytes=n * size + case["rows"] * (8 * case["topk"] + 8 * case["given"] + 4), flops=5 * n)
    sh, page = _shapes(case), case["page"]
    new, past = sh["new"], sh["past"]
    if case["op"] == "pages":
        held = sum(-(-p // page) for p in past)
        grown = sum(-(-(p + n) // page) - -(-p // page) for p, n in zip(past, new))
        pool = held + grown + case["spare"]
        return dict(bytes=4 * (pool + held + 4 * grown) + 12 * sum(new), flops=pool + held)
    d, H = case["dim"], case["kv_heads"]
    if case["op"] == "bounds":
        done = sum((p + n) // page - p // page for p, n in zip(past, new)) * H * case["layers"]
        return dict(bytes=done * (page * (d // 2 + d // 32) + 4 * d), flops=2 * done * page * d)
    size, G = (2 if case["dtype"] == "bf16" else 4), case["heads"] // H
    packed = d + d // 16  # bytes of a key and its value
    nbytes, flops = 2 * sum(new) * case["heads"] * d * size, 0
    for b, (n, p) in enumerate(zip(new, past)):
        full = p // page
        k, tail = min(case["top"], full), p - full * page
        groups = _groups(n, case["share"])
        nbytes += H * ((full * 4 * d if full > case["top"] else 0) +
                       (min(len(groups) * k, full) * page + tail + n) * packed)
        if full > case["top"]:
            flops += 4 * d * n * case["heads"] * full
        own_pairs = sum(x + 1 for x in _depths(sh["trees"][b])) if case["op"] == "tree" else n * (n + 1) // 2
        flops += 4 * d * case["heads"] * (n * (k * page + tail) + own_pairs)
    return dict(bytes=nbytes, flops=flops)


# ----------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------

def _gen(seed, stream):
    g = torch.Generator(device=DEV)
    g.manual_seed((seed * 1000003 + stream) % (1 << 62))
    return g


def _offsets(new):
    o = [0]
    for n in new:
        o.append(o[-1] + n)
    return o


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    st = dict(case=case)
    if case["op"] == "logprobs":
        _prepare_logits(st, case, seed)
    else:
        sh = _shapes(case)
        st.update(sh=sh, offs=_offsets(sh["new"]))
        st.update(offsets=_i32(st["offs"]))
        (_prepare_pages if case["op"] == "pages" else _prepare_cache)(st, case, sh, seed)
    if own:
        _bind(st)
    return st


def _prepare_logits(st, case, seed):
    N, V = case["rows"], case["vocab"]
    g = _gen(seed, 1)
    stride = V + case["pad"]
    # some likely tokens over a long tail, as a trained model's rows are
    K = min(V, 12)
    logits = torch.empty((N, stride), dtype=DTYPES[case["dtype"]], device=DEV)
    cand = torch.randint(0, V, (N, K), generator=g, device=DEV)
    top = math.log(V) + 4.0 + torch.randn((N, K), generator=g, device=DEV) - 0.8 * torch.arange(K, device=DEV)
    for r0 in range(0, N, 64):
        r1 = min(N, r0 + 64)
        x = 2.0 * torch.randn((r1 - r0, stride), generator=g, device=DEV)
        x[:, V:] = 50.0  # padding columns hold anything
        x.scatter_(1, cand[r0:r1], top[r0:r1])
        if case["banned"]:
            ban = torch.randint(0, V, (r1 - r0, case["banned"]), generator=g, device=DEV)
            x.scatter_(1, ban, -math.inf)
        logits[r0:r1] = x.to(logits.dtype)
    tokens = torch.randint(0, V, (N, max(case["given"], 1)), generator=g, device=DEV)
    likely = torch.rand(tokens.shape, generator=g, device=DEV) < 0.7
    tokens = torch.where(likely, cand[:, :1].expand_as(tokens), tokens)
    st.update(logits=logits, given=tokens[:, :case["given"]].int().contiguous())


def _tables(past, new, page, spare, seed):
    """Page tables whose sequences hold scattered pages for `past` tokens, room for the new ones,
    and how many tables hold each page of the pool."""
    held = [-(-p // page) for p in past]
    grown = [-(-(p + n) // page) for p, n in zip(past, new)]
    n_pages, width = sum(grown) + spare, max(grown) + 1
    order = np.random.default_rng(seed * 11 + 5).permutation(n_pages).astype(np.int32)
    table = np.full((len(past), width), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    refs = np.zeros(n_pages, dtype=np.int32)
    refs[order[:at]] = 1
    return table, refs, order, at


def _prepare_pages(st, case, sh, seed):
    spare = case["spare"]
    table, refs, _, _ = _tables(sh["past"], sh["new"], case["page"], spare, seed)
    S, T = case["seqs"], st["offs"][-1]
    st.update(pages=torch.from_numpy(table).to(DEV), refs=torch.from_numpy(refs).to(DEV), length=_i32(sh["past"]),
              missing=torch.empty(S, dtype=torch.int32, device=DEV),
              slots=torch.empty(T, dtype=torch.int64, device=DEV),
              positions=torch.empty(T, dtype=torch.int32, device=DEV),
              # the step accepts nothing: what it took goes back, and the next pass finds the tables as they were
              keep=_i32(sh["past"]),
              depth=_i32([x for t in sh["trees"] for x in _depths(t)]) if "trees" in sh else None)


def _prepare_cache(st, case, sh, seed):
    S, H, d, page = case["seqs"], case["kv_heads"], case["dim"], case["page"]
    Ly = case.get("layers", 1)
    g = _gen(seed, 2)
    table, _, order, at = _tables(sh["past"], sh["new"], page, 3, seed)
    for b in range(S):  # the new tokens' pages too
        lo, hi = -(-sh["past"][b] // page), -(-(sh["past"][b] + sh["new"][b]) // page)
        table[b, lo:hi] = order[at:at + hi - lo]
        at += hi - lo
    n_pages = len(order)
    u8 = dict(dtype=torch.uint8, device=DEV)
    cache = dict(k_codes=torch.empty((Ly, n_pages, H, page * d // 2), **u8),
                 k_scales=torch.empty((Ly, n_pages, H, page * d // 32), **u8),
                 v_codes=torch.empty((Ly, n_pages, H, page * d // 2), **u8),
                 v_scales=torch.empty((Ly, n_pages, H, page * d // 32), **u8),
                 pages=torch.from_numpy(table).to(DEV), length=_i32(sh["past"]))
    # every page of the pool is filled; keys have a few strong channels, as trained projections do, and
    # the tokens of a page have something in common
    gain = torch.exp(0.5 * torch.randn((H, 1, d), generator=g, device=DEV))
    bounds = torch.zeros((Ly, n_pages, H, 2, d), dtype=torch.bfloat16, device=DEV)
    step = max(1, (1 << 26) // (H * page * d))
    for l in range(Ly):
        for p0 in range(0, n_pages, step):
            n = min(n_pages, p0 + step) - p0
            k = torch.randn((n, H, page, d), generator=g, device=DEV)
            k = (k + 0.7 * torch.randn((n, H, 1, d), generator=g, device=DEV)) * gain
            kc, ks = _encode(k)
            cache["k_codes"][l, p0:p0 + n] = (_halves(kc).view(n, H, page // 16, 16, d // 32, 16)
                                              .transpose(3, 4).reshape(n, H, -1))
            cache["k_scales"][l, p0:p0 + n] = ks.reshape(n, H, -1)
            if case["op"] == "bounds":
                continue
            v = torch.randn((n, H, page, d), generator=g, device=DEV)
            vc, vs = _encode(v)
            # token 8 qp + 4 h + t of a group: [group][qp][h][t][m][d/64] to [group][h][m][qp][t][d/64]
            cache["v_codes"][l, p0:p0 + n] = (_halves(vc).view(n, H, page // 16, 2, 2, 4, 32, d // 64)
                                              .permute(0, 1, 2, 4, 6, 3, 5, 7).reshape(n, H, -1))
            cache["v_scales"][l, p0:p0 + n] = (vs.view(n, H, page // 16, 2, 2, 4, d // 32)
                                               .permute(0, 1, 2, 4, 6, 3, 5).reshape(n, H, -1))
            kd = _decode(kc, ks)
            bounds[l, p0:p0 + n] = torch.stack((kd.amax(2), kd.amin(2)), 2).to(torch.bfloat16)
    st.update(cache=cache, bounds=bounds)
    T = st["offs"][-1]
    if case["op"] == "bounds":  # the tokens have been committed
        cache["length"] += _i32(sh["new"])
        return
    st["q"] = (1.5 * torch.randn((1, T, case["heads"], d), generator=g, device=DEV)).to(DTYPES[case["dtype"]])
    st["selected"] = torch.full((1, T, H, case["top"]), -1, dtype=torch.int32, device=DEV)
    if case["op"] == "tree":
        st["parents"] = [torch.tensor(t, dtype=torch.int64, device=DEV) for t in sh["trees"]]


# ----------------------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------------------

def _encode(x):
    """[..., d] values -> (codes [..., d], scale bytes [..., d/32])."""
    xb = x.float().reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    bits = xb.abs().amax(-1).view(torch.int32)
    e = ((bits >> 23) - 129 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(-125, 125)
    y = torch.ldexp(xb.abs(), -e[..., None])
    code = ((y > 0.25).int() + (y >= 0.75).int() + (y > 1.25).int() + (y >= 1.75).int() +
            (y > 2.5).int() + (y >= 3.5).int() + (y > 5.0).int())
    code = code | (torch.signbit(xb).int() << 3)
    return code.reshape(x.shape).to(torch.uint8), (e + 127).to(torch.uint8)


def _decode(codes, scales):
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=codes.device)
    v = grid[codes.long()].reshape(*scales.shape, 32)
    return torch.ldexp(v, scales.int()[..., None] - 127).reshape(codes.shape)


def _halves(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _unhalves(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _slab_keys(codes, scales, d):
    """[..., page d/2] bytes -> keys [..., page, d] in 32 bits."""
    lead, page = codes.shape[:-1], codes.shape[-1] * 2 // d
    c = _unhalves(codes.view(*lead, page // 16, d // 32, 16, 16)).transpose(-3, -2).reshape(*lead, page, d)
    return _decode(c, scales.view(*lead, page, d // 32))


def _slab_values(codes, scales, d):
    lead, page = codes.shape[:-1], codes.shape[-1] * 2 // d
    k = len(lead)
    c = _unhalves(codes.view(*lead, page // 16, 2, 32, 2, 4, d // 64))
    c = c.permute(*range(k), k, k + 3, k + 1, k + 4, k + 2, k + 5).reshape(*lead, page, d)
    e = scales.view(*lead, page // 16, 2, d // 32, 2, 4)
    e = e.permute(*range(k), k, k + 3, k + 1, k + 4, k + 2).reshape(*lead, page, d // 32)
    return _decode(c, e)


def _plain_logprobs(st):
    case, logits = st["case"], st["logits"]
    N, V, K = case["rows"], case["vocab"], case["topk"]
    index = torch.arange(V, device=DEV)
    parts = []
    step = max(1, (1 << 25) // V)
    for r0 in range(0, N, step):
        x = logits[r0:r0 + step, :V].float()
        m = x.amax(1, keepdim=True)
        w = torch.exp(x - m)
        z = w.sum(1, keepdim=True)
        logz = torch.log(z)
        away = torch.where(w > 0, m - x, torch.zeros_like(x))
        out = [(logz + (w * away).sum(1, keepdim=True) / z)[:, 0]]
        # order by value, then by index: one integer for both
        if K:
            bits = x.view(torch.int32).long()
            key = (torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) << 32) + (V - 1 - index)
            top = torch.topk(key, K, dim=1).indices
            out += [top.int(), x.gather(1, top) - m - logz]
        if case["given"]:
            out.append(x.gather(1, st["given"][r0:r0 + step].long()) - m - logz)
        parts.append(out)
    return tuple(torch.cat(p) for p in zip(*parts))


def _ragged(counts):
    """(sequence, index within it) of every row of a ragged batch."""
    seq = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts)).to(DEV)
    idx = torch.cat([torch.arange(n) for n in counts]).to(DEV)
    return seq, idx


def _plain_pages(st):
    case, pages, refs, length = st["case"], st["pages"], st["refs"], st["length"].long()
    page, n_pages = case["page"], refs.numel()
    S, width = pages.shape
    new = (st["offsets"][1:] - st["offsets"][:-1]).long()
    entry = torch.arange(width, device=DEV)
    # reserve
    need = ((length + new + page - 1) // page).clamp(max=width)
    want = (entry < need[:, None]) & ((pages < 0) | (pages >= n_pages))
    order = (want.flatten().cumsum(0) - 1).view(S, width)
    free = refs == 0
    rank = free.long().cumsum(0) - 1
    ids = torch.zeros(n_pages + 1, dtype=torch.int32, device=DEV)
    ids.scatter_(0, torch.where(free, rank, n_pages), torch.arange(n_pages, dtype=torch.int32, device=DEV))
    got = want & (order < free.sum())
    refs.masked_fill_(free & (rank < want.sum()), 1)
    pages.copy_(torch.where(got, ids[order.clamp(0, n_pages)], pages))
    st["missing"].copy_((want & ~got).sum(1))
    seq, idx = _ragged(st["sh"]["new"])
    at = length[seq] + idx
    pid = pages[seq, (at // page).clamp(max=width - 1)].long()
    there = (at // page < width) & (pid >= 0) & (pid < n_pages)
    st["slots"].copy_(torch.where(there, pid * page + at % page, -1))
    st["positions"].copy_(length[seq] + (idx if st["depth"] is None else st["depth"]))
    # release
    drop = entry >= ((st["keep"].long() + page - 1) // page)[:, None]
    back = drop & (pages >= 0) & (pages < n_pages)
    fall = torch.zeros(n_pages + 1, dtype=torch.int32, device=DEV)
    fall.scatter_add_(0, torch.where(back, pages.long(), n_pages).flatten(), torch.ones_like(pages).flatten())
    refs.copy_((refs - fall[:n_pages]).clamp(min=0))
    pages.masked_fill_(drop, -1)
    return st["slots"], st["positions"], st["missing"], pages, refs


def _plain_bounds(st):
    case, cache, bounds = st["case"], st["cache"], st["bounds"]
    page, d = case["page"], case["dim"]
    ids = [cache["pages"][b, p // page:(p + n) // page] for b, (p, n) in enumerate(zip(st["sh"]["past"], st["sh"]["new"]))]
    ids = torch.cat(ids).long()
    for l in range(case["layers"]):
        step = max(1, (1 << 26) // (case["kv_heads"] * page * d))
        for i in range(0, len(ids), step):
            at = ids[i:i + step]
            k = _slab_keys(cache["k_codes"][l, at], cache["k_scales"][l, at], d)
            bounds[l, at] = torch.stack((k.amax(2), k.amin(2)), 2).to(bounds.dtype)
    return bounds


def _plain_select(st, b):
    """Positions in sequence b's page table [groups, kv heads, selected], ascending."""
    case = st["case"]
    H, d, page, top = case["kv_heads"], case["dim"], case["page"], case["top"]
    n, at = st["sh"]["new"][b], st["offs"][b]
    full = st["sh"]["past"][b] // page
    groups = _groups(n, case["share"])
    if full <= top:
        return torch.arange(full, device=DEV).expand(len(groups), H, full)
    lim = st["bounds"][0, st["cache"]["pages"][b, :full].long()].double()  # [full, H, 2, d]
    lim = lim.permute(1, 2, 3, 0).reshape(H, 2 * d, full)
    out = []
    for i0, i1 in groups:
        # near pages differ by less than 32 bits resolve
        x = st["q"][0, at + i0:at + i1].double().view(i1 - i0, H, -1, d).transpose(0, 1).reshape(H, -1, d)
        s = torch.matmul(torch.cat((x.clamp(min=0), x.clamp(max=0)), -1), lim).amax(1)
        s[:, :case["first"]] = math.inf
        s[:, full - case["last"]:] = math.inf
        out.append(torch.sort(s, dim=1, descending=True, stable=True).indices[:, :top].sort(1).values)
    return torch.stack(out)


def _plain_sparse(st):
    case, cache, q = st["case"], st["cache"], st["q"]
    Hq, H, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    G = Hq // H
    out = torch.empty_like(q)
    head = torch.arange(H, device=DEV)[:, None]
    for b in range(case["seqs"]):
        n, past, at = st["sh"]["new"][b], st["sh"]["past"][b], st["offs"][b]
        full = past // page
        sel = _plain_select(st, b)
        K = sel.shape[2]
        table = cache["pages"][b].long()
        if case["op"] == "tree":
            vis = torch.zeros((n, n), dtype=torch.bool, device=DEV)
            rows = torch.arange(n, device=DEV)
            cur = rows
            for _ in range(case["depth"] + 1):
                vis[rows, cur.clamp(min=0)] |= cur >= 0
                cur = torch.where(cur >= 0, st["parents"][b][cur.clamp(min=0)], cur)
        else:
            vis = torch.ones((n, n), dtype=torch.bool, device=DEV).tril()
        for k, (i0, i1) in enumerate(_groups(n, case["share"])):
            st["selected"][0, at + i0, :, :K] = sel[k].int()
            end = past + (n if case["op"] == "tree" else i1)
            tail = torch.arange(full, -(-end // page), device=DEV)
            ids = table[torch.cat((sel[k], tail.expand(H, -1)), 1)]  # [H, pages]
            L = K * page + end - full * page
            kk = _slab_keys(cache["k_codes"][0][ids, head], cache["k_scales"][0][ids, head], d)
            vv = _slab_values(cache["v_codes"][0][ids, head], cache["v_scales"][0][ids, head], d)
            kk, vv = kk.view(H, -1, d)[:, :L], vv.view(H, -1, d)[:, :L]
            x = q[0, at + i0:at + i1].float().view(i1 - i0, H, G, d).transpose(0, 1).reshape(H, -1, d)
            s = torch.matmul(x * d ** -0.5, kk.transpose(1, 2).contiguous()).view(H, i1 - i0, G, L)
            s[..., L - (end - past):].masked_fill_(~vis[i0:i1, None, :end - past], -math.inf)
            p = torch.exp(s - s.amax(-1, keepdim=True))
            o = torch.matmul(p.view(H, -1, L), vv).view(H, i1 - i0, G, d) / p.sum(-1, keepdim=True)
            out[0, at + i0:at + i1] = o.transpose(0, 1).reshape(i1 - i0, Hq, d).to(q.dtype)
    return out, st["selected"]


# ----------------------------------------------------------------------------------------
# the framework's calls
# ----------------------------------------------------------------------------------------

def _bind(st):
    """The handle, plan and buffers that a serving program keeps between calls."""
    from gated_deltanet_tree_amd import binding
    case = st["case"]

    def scratch(nbytes):
        return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=DEV)

    if case["op"] == "logprobs":
        N, V, K = case["rows"], case["vocab"], case["topk"]
        f32 = dict(dtype=torch.float32, device=DEV)
        st.update(entropy=torch.empty(N, **f32), top_logp=torch.empty((N, K), **f32) if K else None,
                  top_token=torch.empty((N, K), dtype=torch.int32, device=DEV) if K else None,
                  given_logp=torch.empty((N, case["given"]), **f32) if case["given"] else None,
                  ws=scratch(binding.logprobs_workspace_bytes(N, V, K)))
        st["args"] = binding.logprobs_args(st["logits"], vocab=V, given=st["given"] if case["given"] else None,
                                           given_logp=st["given_logp"], top_token=st["top_token"],
                                           top_logp=st["top_logp"], entropy=st["entropy"], workspace=st["ws"])
        return
    st["host_offs"] = np.array(st["offs"], dtype=np.int32)
    if case["op"] == "pages":
        kw = dict(missing=st["missing"], slots=st["slots"], positions=st["positions"], depth=st["depth"])
        args = (st["pages"], st["length"], st["refs"], case["page"], st["host_offs"], st["offsets"])
        st["ws"] = scratch(binding.pages_workspace_bytes(binding.pages_args(*args, **kw)))
        st["args"] = binding.pages_args(*args, workspace=st["ws"], **kw)
        return
    kv = binding.KvCache(page_tokens=case["page"], **st["cache"])
    if case["op"] == "bounds":
        st["args"] = binding.kv_args(kv, st["host_offs"], st["offsets"], n_layers=case["layers"])
        st["sparse"] = binding.sparse_args(st["args"], bounds=st["bounds"])
        return
    st["out"] = torch.empty_like(st["q"])
    longest = max(p + n for p, n in zip(st["sh"]["past"], st["sh"]["new"]))
    kw = dict(q=st["q"], out=st["out"], max_length=longest)

    def sparse(a):
        return binding.sparse_args(a, bounds=st["bounds"], selected=st["selected"], top_pages=case["top"],
                                   share_tokens=case["share"], keep_first=case["first"], keep_last=case["last"])

    a = binding.kv_args(kv, st["host_offs"], st["offsets"], **kw)
    st["ws"] = scratch(binding.sparse_workspace_bytes(a, sparse(a)))
    st["args"] = binding.kv_args(kv, st["host_offs"], st["offsets"], workspace=st["ws"], **kw)
    st["sparse"] = sparse(st["args"])
    if case["op"] == "tree":
        st["image"] = binding.hld_schedule([np.array(t, dtype=np.int32) for t in st["sh"]["trees"]])
        st["dev_image"] = torch.from_numpy(st["image"]).to(DEV)


def _own(st):
    from gated_deltanet_tree_amd import binding
    case = st["case"]
    if case["op"] == "logprobs":
        binding.token_logprobs(st["args"])
        return tuple(st[k] for k in ("entropy", "top_token", "top_logp", "given_logp") if st[k] is not None)
    if case["op"] == "pages":
        binding.kv_reserve(st["args"])
        binding.kv_release(st["args"], st["keep"])
        return st["slots"], st["positions"], st["missing"], st["pages"], st["refs"]
    if case["op"] == "bounds":
        binding.kv_bounds(st["args"], st["sparse"])
        return st["bounds"]
    binding.kv_select(st["args"], st["sparse"])
    if case["op"] == "tree":
        binding.sparse_tree_attention(st["args"], st["sparse"], st["image"], st["dev_image"])
    else:
        binding.sparse_attention(st["args"], st["sparse"])
    return st["out"], st["selected"]


def run(state):
    if own:
        return _own(state)
    return {"logprobs": _plain_logprobs, "pages": _plain_pages, "bounds": _plain_bounds, "sparse": _plain_sparse,
            "tree": _plain_sparse}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------------------
# the operators' definitions in 64 bits
# ----------------------------------------------------------------------------------------

def _exact_logprobs(case, st):
    V, K = case["vocab"], case["topk"]
    ent, tok, top, giv = [], [], [], []
    for r in range(case["rows"]):
        x = st["logits"][r, :V].double()
        logp = x - torch.logsumexp(x, 0)
        p = torch.exp(logp)
        ent.append(-(p * torch.where(p > 0, logp, torch.zeros_like(p))).sum())
        if K:
            vals, order = torch.sort(x, descending=True, stable=True)
            tok.append(order[:K].int())
            top.append(logp[order[:K]])
        if case["given"]:
            giv.append(logp[st["given"][r].long()])
    return tuple(torch.stack(x) for x in (ent, tok, top, giv) if x)


def _exact_pages(case, st):
    page = case["page"]
    table, refs = st["pages"].cpu().numpy().copy(), st["refs"].cpu().numpy().copy()
    S, width = table.shape
    free = iter(np.flatnonzero(refs == 0).tolist())
    missing, slots, positions = [], [], []
    for b, (n, p) in enumerate(zip(st["sh"]["new"], st["sh"]["past"])):
        short = 0
        for i in range(min(width, -(-(p + n) // page))):
            if not 0 <= table[b, i] < len(refs):
                got = next(free, None)
                if got is None:
                    short += 1
                else:
                    table[b, i], refs[got] = got, 1
        missing.append(short)
        dep = _depths(st["sh"]["trees"][b]) if "trees" in st["sh"] else range(n)
        for i in range(n):
            k = (p + i) // page
            slots.append(int(table[b, k]) * page + (p + i) % page if k < width and table[b, k] >= 0 else -1)
            positions.append(p + dep[i])
    for b, p in enumerate(st["sh"]["past"]):
        for i in range(-(-p // page), width):
            if 0 <= table[b, i] < len(refs):
                refs[table[b, i]] = max(0, refs[table[b, i]] - 1)
            table[b, i] = -1
    return (torch.tensor(slots, device=DEV), _i32(positions), _i32(missing), torch.from_numpy(table).to(DEV),
            torch.from_numpy(refs).to(DEV))


def _bytes_at(pool, base, off):
    return pool.reshape(-1)[base[:, None] + off].long()


def _exact_slots(case, cache, layer, head, page_id, t):
    """Keys and values [n, d] of slots t of pages page_id in 64 bits, by byte address (values: None
    where there are none)."""
    d, H, page = case["dim"], case["kv_heads"], case["page"]
    slab = (layer * cache["k_codes"].shape[1] + page_id.long()) * H + head
    sub, t = t // 16, t % 16
    c = torch.arange(d, device=DEV)
    signed = torch.tensor([*GRID, *(-x for x in GRID)], dtype=torch.float64, device=DEV)
    two = torch.tensor(2.0, dtype=torch.float64, device=DEV)
    code_base, scale_base = slab * (page * d // 2) + sub * 8 * d, slab * (page * d // 32) + sub * (d // 2)
    kb = _bytes_at(cache["k_codes"], code_base + 16 * t, (c // 32) * 256 + (c % 32) // 2)
    ks = _bytes_at(cache["k_scales"], scale_base + t * (d // 32), c // 32)
    k = signed[(kb >> (4 * (c & 1))) & 15] * torch.pow(two, (ks - 127).double())
    if case["op"] == "bounds":
        return k, None
    quad = t // 4
    m, nib = c // (d // 32), c % (d // 32)
    vb = _bytes_at(cache["v_codes"],
                   code_base + (quad % 2) * 4 * d + (quad // 2) * (d // 16) + (t % 4) * (d // 64),
                   m * (d // 8) + nib // 2)
    vs = _bytes_at(cache["v_scales"],
                   scale_base + (quad % 2) * (d // 4) + (quad // 2) * 4 + t % 4, (c // 32) * 8)
    return k, signed[(vb >> (4 * (nib & 1))) & 15] * torch.pow(two, (vs - 127).double())


def _exact_bounds(case, st):
    cache, page, d = st["cache"], case["page"], case["dim"]
    out = st["bounds"].double()
    t = torch.arange(page, device=DEV)
    for b, (p, n) in enumerate(zip(st["sh"]["past"], st["sh"]["new"])):
        ids = cache["pages"][b, p // page:(p + n) // page].long()
        for l in range(case["layers"]):
            for h in range(case["kv_heads"]):
                k, _ = _exact_slots(case, cache, l, h, ids.repeat_interleave(page), t.repeat(len(ids)))
                k = k.view(len(ids), page, d)
                out[l, ids, h, 0], out[l, ids, h, 1] = k.max(1).values, k.min(1).values
    return out


def _exact_sparse(case, st):
    d, H, page = case["dim"], case["kv_heads"], case["page"]
    G = case["heads"] // H
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    chosen = np.full(tuple(st["selected"].shape), -1, dtype=np.int32)
    for b in range(case["seqs"]):
        n, past, at = st["sh"]["new"][b], st["sh"]["past"][b], st["offs"][b]
        full = past // page
        see = torch.zeros((n, n), dtype=torch.bool)
        for i in range(n):
            if case["op"] == "tree":
                p = st["sh"]["trees"][b][i]
                if p >= 0:
                    see[i] = see[p]
                see[i, i] = True
            else:
                see[i, :i + 1] = True
        see = see.to(DEV)
        table = st["cache"]["pages"][b].long()
        for h in range(H):
            qh = st["q"][0, at:at + n, h * G:(h + 1) * G].double()
            slot = torch.arange(past + n, device=DEV)
            k, v = _exact_slots(case, st["cache"], 0, h, table[slot // page], slot % page)
            # the keys themselves give the pages' limits
            kp = k[:full * page].view(full, page, d) if full else None
            for i0, i1 in _groups(n, case["share"]):
                if full > case["top"]:
                    x = qh[i0:i1].reshape(-1, 1, d)
                    hi, lo = kp.max(1).values, kp.min(1).values
                    s = torch.stack([torch.maximum(r * hi, r * lo).sum(1) for r in x]).max(0).values.cpu().numpy()
                    s[:case["first"]] = np.inf
                    s[full - case["last"]:] = np.inf
                    sel = np.sort(np.lexsort((np.arange(full), -s))[:case["top"]])
                else:
                    sel = np.arange(full)
                chosen[0, at + i0, h, :len(sel)] = sel
                use = torch.zeros(past + n, dtype=torch.bool, device=DEV)
                use[:full * page].view(full, page)[torch.from_numpy(sel).to(DEV)] = True
                use[full * page:] = True
                idx = use.nonzero()[:, 0]
                ok = torch.ones((i1 - i0, past + n), dtype=torch.bool, device=DEV)
                ok[:, past:] = see[i0:i1]
                s = torch.matmul(qh[i0:i1].reshape(-1, d), k[idx].T.contiguous()) / math.sqrt(d)
                s = s.masked_fill(~ok[:, idx].repeat_interleave(G, 0), -math.inf)
                o = torch.matmul(torch.softmax(s, -1), v[idx])
                out[0, at + i0:at + i1, h * G:(h + 1) * G] = o.view(i1 - i0, G, d)
    return out, torch.from_numpy(chosen).to(DEV)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("sparse", "tree"):
        # a row loop over scores and long contexts
        rows = sum(st["sh"]["new"]) * case["heads"]
        groups = sum(len(_groups(n, case["share"])) for n in st["sh"]["new"]) * case["kv_heads"]
        if rows > 60000 or groups > 4000:
            return None
        return _exact_sparse(case, st)
    return {"logprobs": _exact_logprobs, "pages": _exact_pages, "bounds": _exact_bounds}[case["op"]](case, st)
