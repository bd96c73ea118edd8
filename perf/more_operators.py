"""Measured cases of attention with shaped scores, block-scaled caches and rotation by several axes.

  attend  attention of new tokens over the paged cache, from one token a
          request to whole prompts, whose scores are capped by a tanh or get a
          bias by distance, and whose tokens each see an interval of positions
          (windows, documents, prefixes, image spans); over bf16 caches, or
          over E4M3 codes with a power-of-two scale per block and head;
  mrope   per-head RMS norm of q and k, rotation by positions of several axes,
          and the write of k and v into the paged cache;
  append  the like into a block-scaled cache: the scale of a block covers all
          its positions, and grows with those that are appended.

`run` takes what `prepare` made through one pass of one operator: with `own`
false by elementary torch operations in 32 bits, with `own` true through the
package.  `exact` restates the definitions in 64 bits.
"""

import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the smallest attention step: ragged new tokens of four requests, small heads, a bias by distance
        dict(name="attend 4 requests alibi d64", op="attend", seqs=4, new=3, even=False, hq=4, hkv=2, d=64, block=16,
             shortest=4, longest=37, cap=0.0, alibi=True, mask="causal", span=0, scaled=False),
        # one decode step of the 8B-shaped batch, a model that caps its scores
        dict(name="attend 64 decodes capped", op="attend", seqs=64, new=1, even=True, hq=32, hkv=8, d=128, block=16,
             shortest=512, longest=4096, cap=50.0, alibi=False, mask="causal", span=0, scaled=False),
        # one decode step of such a model's windowed layers, ragged lengths
        dict(name="attend 96 windowed decodes", op="attend", seqs=96, new=1, even=True, hq=32, hkv=4, d=128, block=32,
             shortest=100, longest=8000, cap=30.0, alibi=False, mask="window", span=1024, scaled=False),
        # whole prompts with images, whose positions see one another whole
        dict(name="attend 8 prompts with spans", op="attend", seqs=8, new=2003, even=True, hq=32, hkv=8, d=128, block=16,
             shortest=2003, longest=2003, cap=50.0, alibi=False, mask="spans", span=300, scaled=False),
        # documents packed into ragged prompts, some rows padding: every head has keys of its own, and small
        dict(name="attend 6 of documents alibi", op="attend", seqs=6, new=1501, even=False, hq=16, hkv=16, d=64, block=32,
             shortest=700, longest=1700, cap=0.0, alibi=True, mask="documents", span=411, scaled=False),
        # the decode step again, on a block-scaled cache
        dict(name="attend 64 decodes scaled", op="attend", seqs=64, new=1, even=True, hq=32, hkv=8, d=128, block=16,
             shortest=512, longest=4096, cap=0.0, alibi=False, mask="causal", span=0, scaled=True),
        # verification of eight tokens over long contexts: the keys have to be split over the whole device
        dict(name="attend 8 long verify 8 scaled", op="attend", seqs=8, new=8, even=True, hq=32, hkv=8, d=128, block=32,
             shortest=32000, longest=32768, cap=0.0, alibi=False, mask="causal", span=0, scaled=True),
        # prompt chunks over cached prefixes
        dict(name="attend 8 chunks scaled", op="attend", seqs=8, new=512, even=True, hq=32, hkv=8, d=128, block=16,
             shortest=2048, longest=8192, cap=0.0, alibi=False, mask="causal", span=0, scaled=True),
        # a few requests decoding: latency
        dict(name="mrope 6 tokens", op="mrope", tokens=6, pad=0, hq=32, hkv=8, d=128, sections="16 24 24", shuffled=False,
             interleaved=False, norm=True, block=16, longest=4096, chunk=1),
        # prompt chunks with images, the axes taking pairs in turn
        dict(name="mrope 5003 tokens", op="mrope", tokens=5003, pad=0, hq=32, hkv=4, d=128, sections="24 20 20",
             shuffled=True, interleaved=False, norm=False, block=32, longest=32768, chunk=617),
        # a padded decode batch: codes of blocks whose scale grows are coded again
        dict(name="append 250 of 256 tokens", op="append", tokens=256, pad=6, hq=32, hkv=8, d=128, sections="64",
             shuffled=False, interleaved=False, norm=True, block=16, longest=32768, chunk=1),
        # sixteen whole prompts at once, with images
        dict(name="append 32048 tokens", op="append", tokens=32048, pad=0, hq=32, hkv=8, d=128, sections="16 24 24",
             shuffled=False, interleaved=False, norm=True, block=16, longest=4096, chunk=2003),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "mrope", "append"])
    block = rng.choice([8, 16, 32])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8])
    if op != "attend":
        d = rng.choice([64, 128])
        tokens = _log_int(rng, 1, 16000)
        half = rng.choice([16, d // 2, d // 2]) if d == 64 else rng.choice([32, 64, 64])
        t = rng.randint(1, half - 2)
        h = rng.randint(1, half - t - 1)
        sections = rng.choice(["%d" % half, "%d %d %d" % (t, h, half - t - h), "%d %d %d" % (half - 2 * (half // 8 * 3), half // 8 * 3, half // 8 * 3)])
        return dict(op=op, tokens=tokens, pad=rng.randint(0, tokens // 8), hq=hq, hkv=hkv, d=d, sections=sections,
                    shuffled=rng.random() < 0.4, interleaved=rng.random() < 0.3, norm=rng.random() < 0.7, block=block,
                    longest=_log_int(rng, 2000, 131072), chunk=_log_int(rng, max(1, tokens // 250), 600))
    scaled = rng.random() < 0.5
    new = rng.choice([1, 1, _log_int(rng, 2, 64), _log_int(rng, 65, 1500)])
    longest = max(_log_int(rng, 40, 20000), new)
    if new > 64:
        longest = min(longest, max(new, 4000))
    most = min(200, 200000 // longest, 700_000_000 // (longest * hq * new))      # no dearer than the listed ones
    mask = rng.choice(["causal", "window", "documents", "spans"])
    return dict(op="attend", seqs=_log_int(rng, 1, max(1, most)), new=new, even=rng.random() < 0.3, hq=hq, hkv=hkv,
                d=128 if scaled else rng.choice([64, 128]), block=block, shortest=max(1, longest // rng.choice([1, 4, 20])),
                longest=longest, cap=rng.choice([0.0, 0.0, 20.0, 50.0]), alibi=rng.random() < 0.3, mask=mask,
                span=0 if mask == "causal" else _log_int(rng, 16, 3000), scaled=scaled)


# ---------------------------------------------------------------------------
# sizes that follow from a case alone (the seed only orders them)
# ---------------------------------------------------------------------------

def _attend_sizes(case):
    """(context length, new tokens) of each request, in a fixed order."""
    S, m = case["seqs"], case["new"]
    u = (np.arange(S) + 0.5) / S
    ctx = np.round(case["shortest"] + u * (case["longest"] - case["shortest"])).astype(np.int64)
    new = np.full(S, m) if case["even"] else 1 + (np.arange(S) * 7 + m - 1) % m
    return ctx, np.minimum(new, ctx)


def _visible(case, ctx, new):
    """[new, 2]: the interval of positions that each new token of a request sees."""
    p = np.arange(ctx - new, ctx)
    lo, hi, span = np.zeros_like(p), p + 1, case["span"]
    if case["mask"] == "window":
        lo = np.maximum(0, p - span + 1)
    elif case["mask"] == "documents":                    # one document after another; some rows are padding
        lo = p // span * span
        hi = np.where((p % 29 == 28) & (new > 1), lo, hi)
    elif case["mask"] == "spans":                        # image, text, image, ...: an image's positions see all of it
        hi = np.where(p // span % 2 == 0, np.minimum((p // span + 1) * span, ctx), hi)
    return np.stack([lo, hi], 1).astype(np.int32)


def _runs(case):
    """Tokens of the runs of consecutive positions that make up the tokens."""
    left, runs = case["tokens"] - case["pad"], []
    while left > 0:
        runs.append(min(case["chunk"], left))
        left -= runs[-1]
    return runs


def work(case):
    if case["op"] != "attend":
        T, half = case["tokens"] - case["pad"], sum(int(x) for x in case["sections"].split())
        axes = len(case["sections"].split())
        q, kv = case["hq"] * case["d"], 2 * case["hkv"] * case["d"]
        n = T * (4 * q + 2 * kv + (2 * kv if case["op"] == "mrope" else kv) + 4 * axes + 8) + 8 * half * min(T, case["longest"])
        if case["op"] == "append":
            n += 4 * case["hkv"] * sum(-(-r // case["block"]) for r in _runs(case))
        return {"bytes": n, "flops": T * (q + kv // 2) * 8}
    seen = read = blocks = tokens = 0
    for c, n in zip(*_attend_sizes(case)):
        v = _visible(case, int(c), int(n)).astype(np.int64)
        some = np.maximum(v[:, 1] - v[:, 0], 0)
        seen += int(some.sum())
        edge = np.zeros(int(c) + 1, dtype=np.int64)
        np.add.at(edge, v[some > 0, 0], 1)
        np.add.at(edge, v[some > 0, 1], -1)
        any_ = np.cumsum(edge)[:-1] > 0
        read += int(any_.sum())
        blocks += int(np.add.reduceat(any_, np.arange(0, int(c), case["block"])).astype(bool).sum())
        tokens += int(n)
    kv = 2 * read * case["hkv"] * case["d"] * (1 if case["scaled"] else 2)
    kv += blocks * (4 + (2 * case["hkv"] if case["scaled"] else 0))
    return {"bytes": kv + 4 * tokens * case["hq"] * case["d"] + (0 if case["mask"] == "causal" else 8 * tokens),
            "flops": 4 * seen * case["hq"] * case["d"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _scaled_cache(shape, g, rng):
    """E4M3 codes and the power-of-two scale of each (block, head), as biased exponents."""
    codes = torch.randn(shape, generator=g, device="cuda").mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, _dev(rng.integers(118, 122, size=shape[:2]).astype(np.uint8))


def _prepare_attend(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    ctx, new = _attend_sizes(case)
    order = rng.permutation(len(ctx))
    ctx, new = ctx[order], new[order]
    hq, hkv, d, B = case["hq"], case["hkv"], case["d"], case["block"]
    blocks = -(-ctx // B)
    NB, MB = int(blocks.sum()) + 5, int(blocks.max())
    ids = rng.permutation(NB)
    tables = np.full((len(ctx), MB), -1, dtype=np.int32)
    at = 0
    for s, b in enumerate(blocks):
        tables[s, :b] = ids[at:at + b]
        at += int(b)
    start = np.concatenate([[0], np.cumsum(new)])
    T = int(start[-1])
    seq = np.repeat(np.arange(len(ctx)), new)
    shape = (NB, hkv, B, d)
    ks = vs = None
    if case["scaled"]:
        kc, ks = _scaled_cache(shape, g, rng)
        vc, vs = _scaled_cache(shape, g, rng)
    else:
        kc, vc = (torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(T, hq, d, generator=g, device="cuda").mul_(2).to(torch.bfloat16)
    visible = np.concatenate([_visible(case, int(c), int(n)) for c, n in zip(ctx, new)])
    slopes = 2.0 ** (-8.0 * np.arange(1, hq + 1) / hq)
    return dict(q=q, kc=kc, vc=vc, k_scales=ks, v_scales=vs, tables=_dev(tables), query_start=_dev(start.astype(np.int32)),
                context_lens=_dev(ctx.astype(np.int32)), visible=None if case["mask"] == "causal" else _dev(visible),
                ranges=_dev(visible), slopes=_dev(slopes.astype(np.float32)) if case["alibi"] else None, cap=case["cap"],
                seq=_dev(seq), nth=_dev(np.arange(T) - start[seq]), new=_dev(new), most_new=case["new"],
                max_ctx=case["longest"], B=B, scale=1 / math.sqrt(d), hq=hq, hkv=hkv, d=d,
                out=torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda"))


def _axes(case):
    """The axis whose position turns each pair: section after section, or the axes in turn while they have pairs left."""
    left = [int(x) for x in case["sections"].split()]
    if not case["shuffled"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    axes = []
    while any(left):
        for a, n in enumerate(left):
            if n:
                axes.append(a)
                left[a] -= 1
    return axes


def _prepare_rope(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    T, hq, hkv, d, B = case["tokens"], case["hq"], case["hkv"], case["d"], case["block"]
    qkv = torch.randn(T, (hq + 2 * hkv) * d, generator=g, device="cuda").mul_(1.5).to(torch.bfloat16)
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    axes, runs, pad = _axes(case), _runs(case), case["pad"]
    A, half = max(axes) + 1, len(axes)
    pos = np.concatenate([np.arange(n) + rng.integers(0, case["longest"] - n + 1) for n in runs])
    where = np.stack([pos] * A)
    if A > 1:                                             # images of 16 x 16 patches between stretches of text
        image = pos // 256 % 2 == 1
        where = np.where(image, np.stack([pos // 256 * 256, pos // 256 * 256 + pos // 16 % 16, pos // 256 * 256 + pos % 16]), where)
    NB = sum(-(-n // B) + 1 for n in runs) + 3
    ids, slots, at = rng.permutation(NB), [], 0
    for n in runs:                                        # each run sits in blocks of its own, from some offset on
        j = np.arange(n) + rng.integers(0, B)
        slots.append(ids[at + j // B] * B + j % B)
        at += -(-n // B) + 1
    slots = np.concatenate(slots + [np.full(pad, -1)]).astype(np.int64)
    positions = np.concatenate([where, np.full((A, pad), -1)], 1).astype(np.int32)
    angle = torch.arange(case["longest"], dtype=torch.float64, device="cuda")[:, None] * \
        10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
    gain = lambda: 1 + 0.1 * torch.randn(d, generator=g, device="cuda")  # noqa: E731
    qw, kw = (gain(), gain()) if case["norm"] else (None, None)
    shape = (NB, hkv, B, d)
    st = dict(q=q, k=k, v=v, positions=_dev(positions), slots=_dev(slots), cos_sin=cos_sin, axes=axes, qw=qw, kw=kw, eps=1e-6,
              axis=_dev(np.array(axes, dtype=np.int64)), n=T - pad, interleaved=case["interleaved"], B=B,
              q_out=torch.zeros(T, hq, d, dtype=torch.bfloat16, device="cuda"))
    if case["op"] == "append":
        kc, ks = _scaled_cache(shape, g, rng)
        vc, vs = _scaled_cache(shape, g, rng)
        st.update(kc=kc, vc=vc, k_scales=ks, v_scales=vs)
    else:
        st.update(kc=torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16),
                  vc=torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16))
    return st


def prepare(case, seed):
    st = (_prepare_attend if case["op"] == "attend" else _prepare_rope)(case, seed)
    st["op"] = case["op"]
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _gathered(cache, scales, tables):
    """A cache's positions in order, [S, Hkv, positions, D] in 32 bits."""
    x = cache[tables.clamp(min=0).long()]
    if scales is None:
        x = x.float()
    else:
        x = x.view(torch.float8_e4m3fn).float() * (scales[tables.clamp(min=0).long()].float() - 127).exp2()[..., None, None]
    S, MB, H, B, D = x.shape
    return x.transpose(1, 2).reshape(S, H, MB * B, D)


def _run_attend(st):
    if own:
        from paged_kv_cache_124_gb300 import api
        if "workspace" not in st:
            st["workspace"] = api.attend_workspace(st["tables"].shape[0], st["most_new"], st["tables"].shape[1], st["B"],
                                                   st["hq"], st["hkv"], st["d"], scaled=st["k_scales"] is not None)
        api.pa_attend(st["out"], st["q"], st["kc"], st["vc"], st["tables"], st["query_start"], st["context_lens"],
                      st["most_new"], st["B"], st["scale"], st["hq"], st["hkv"], st["d"], st["max_ctx"],
                      visible=st["visible"], softcap=st["cap"], slopes=st["slopes"], k_scales=st["k_scales"],
                      v_scales=st["v_scales"], workspace=st["workspace"])
        return st["out"]
    S, m, G = st["tables"].shape[0], st["most_new"], st["hq"] // st["hkv"]
    K = _gathered(st["kc"], st["k_scales"], st["tables"])
    V = _gathered(st["vc"], st["v_scales"], st["tables"])
    i = torch.arange(m, device="cuda")
    at = (st["query_start"][:-1, None] + i).clamp(max=st["q"].shape[0] - 1).long()    # token i of each request
    q = st["q"][at].float().unflatten(2, (st["hkv"], G)).permute(0, 2, 1, 3, 4).reshape(S, st["hkv"], m * G, -1)
    j = torch.arange(K.shape[2], device="cuda")
    lo, hi = st["ranges"][at].unbind(-1)
    seen = (j >= lo[..., None]) & (j < hi[..., None])
    s = (q @ K.transpose(-1, -2)).unflatten(2, (m, G)) * st["scale"]
    if st["cap"]:
        s = (s / st["cap"]).tanh() * st["cap"]
    if st["slopes"] is not None:
        p = (st["context_lens"] - st["new"])[:, None, None] + i[:, None]
        s = s - st["slopes"].view(1, st["hkv"], 1, G, 1) * (p - j).abs()[:, None, :, None]
    s = s.masked_fill(~seen[:, None, :, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    w = (s - torch.where(top > -math.inf, top, 0)).exp()
    total = w.sum(-1, keepdim=True)
    o = w.flatten(2, 3) @ V
    o = o.unflatten(2, (m, G)) / torch.where(total > 0, total, 1)
    o = o.permute(0, 2, 1, 3, 4).flatten(2, 3)                     # [S, m, Hq, D]
    st["out"].copy_(o[st["seq"], st["nth"]])
    return st["out"]


def _rope_outputs(st):
    if st["op"] == "mrope":
        return {"q": st["q_out"], "k_cache": st["kc"], "v_cache": st["vc"]}
    return {"q": st["q_out"], "k_cache": st["kc"].view(torch.float8_e4m3fn), "v_cache": st["vc"].view(torch.float8_e4m3fn),
            "k_scales": st["k_scales"].view(torch.float8_e8m0fnu), "v_scales": st["v_scales"].view(torch.float8_e8m0fnu)}


def _plain_norm_rope(x, gain, eps, cos, sin, interleaved):
    x = x.float()
    if gain is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * gain
    half = cos.shape[-1]
    turn, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = turn[..., :half], turn[..., half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, rest], -1)


def _plain_append(codes, scales, x, blk, off):
    """x [T, Hkv, D] to codes[blk, :, off]; scales cover what a block holds."""
    NB, B = codes.shape[0], codes.shape[2]
    top = torch.zeros(scales.shape, device="cuda").index_reduce_(0, blk, x.abs().amax(-1), "amax")
    part, up = torch.frexp(top)
    need = torch.where(top > 0, up - 9 + (part > 0.875).int(), -127).clamp(min=-127)   # the least e with top <= 448 * 2^e
    first = torch.full((NB,), B, device="cuda").index_reduce_(0, blk, off, "amin")     # the first offset written in a block
    old = scales.int() - 127
    new = torch.where((first == B)[:, None], old, torch.where((first == 0)[:, None], need, torch.maximum(need, old)))
    grown = ((first > 0) & (first < B))[:, None] & (new > old)
    again = codes.view(torch.float8_e4m3fn).float() * torch.where(grown, old - new, 0).float().exp2()[..., None, None]
    codes.copy_(again.to(torch.float8_e4m3fn).view(torch.uint8))
    scales.copy_(new + 127)
    codes[blk, :, off] = (x * (-new[blk].float()).exp2()[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _run_rope(st):
    if own:
        from paged_kv_cache_124_gb300 import api
        if st["op"] == "mrope":
            api.pa_qk_norm_mrope_cache(st["q_out"], st["kc"], st["vc"], st["q"], st["k"], st["v"], st["positions"],
                                       st["axes"], st["slots"], st["cos_sin"], q_weight=st["qw"], k_weight=st["kw"],
                                       eps=st["eps"], interleaved=st["interleaved"])
        else:
            api.pa_qk_norm_rope_cache_scaled(st["q_out"], st["kc"], st["vc"], st["k_scales"], st["v_scales"], st["q"],
                                             st["k"], st["v"], st["positions"], st["slots"], st["cos_sin"],
                                             axes=st["axes"], q_weight=st["qw"], k_weight=st["kw"], eps=st["eps"],
                                             interleaved=st["interleaved"])
        return _rope_outputs(st)
    n, B, half = st["n"], st["B"], st["axis"].shape[0]
    pair = torch.arange(half, device="cuda")
    at = st["positions"][st["axis"], :n].long().T         # [n, half]: the position that turns each pair
    cos, sin = st["cos_sin"][at, pair][:, None], st["cos_sin"][at, half + pair][:, None]
    q = _plain_norm_rope(st["q"][:n], st["qw"], st["eps"], cos, sin, st["interleaved"])
    k = _plain_norm_rope(st["k"][:n], st["kw"], st["eps"], cos, sin, st["interleaved"])
    st["q_out"][:n] = q.to(torch.bfloat16)
    blk, off = st["slots"][:n] // B, st["slots"][:n] % B
    if st["op"] == "mrope":
        st["kc"][blk, :, off] = k.to(torch.bfloat16)
        st["vc"][blk, :, off] = st["v"][:n]
    else:
        _plain_append(st["kc"], st["k_scales"], k, blk, off)
        _plain_append(st["vc"], st["v_scales"], st["v"][:n].float(), blk, off)
    return _rope_outputs(st)


def run(state):
    return (_run_attend if state["op"] == "attend" else _run_rope)(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_attend(case, seed):
    st = _prepare_attend(case, seed)
    G, hkv, d = st["hq"] // st["hkv"], st["hkv"], st["d"]
    start, ctxs = st["query_start"].tolist(), st["context_lens"].tolist()
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for s, C in enumerate(ctxs):
        lo, hi = start[s], start[s + 1]
        n = hi - lo
        ids = st["tables"][s, :-(-C // st["B"])].long()

        def rows(cache, scales):
            x = cache[ids]
            if scales is not None:
                x = torch.ldexp(x.view(torch.float8_e4m3fn).double(), scales[ids].int()[..., None, None] - 127)
            return x.double().permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, :C]

        K, V = rows(st["kc"], st["k_scales"]), rows(st["vc"], st["v_scales"])
        place = torch.arange(C, device="cuda")
        see = (place >= st["ranges"][lo:hi, :1]) & (place < st["ranges"][lo:hi, 1:])
        far = (place - torch.arange(C - n, C, device="cuda")[:, None]).abs().double()
        for h in range(hkv):
            logits = torch.einsum("ngd,cd->gnc", st["q"][lo:hi, h * G:(h + 1) * G].double(), K[h]) * st["scale"]
            if case["cap"]:
                logits = case["cap"] * torch.tanh(logits / case["cap"])
            if case["alibi"]:
                logits = logits - st["slopes"][h * G:(h + 1) * G].double()[:, None, None] * far
            logits = torch.where(see, logits, torch.full_like(logits, -math.inf))
            weights = torch.where(see, torch.softmax(logits, -1), torch.zeros_like(logits))     # a row that sees nothing: zeros
            out[lo:hi, h * G:(h + 1) * G] = torch.einsum("gnc,cd->ngd", weights, V[h])
    return out


def _exact_rope(case, seed):
    st = _prepare_rope(case, seed)
    n, B, d, half = st["n"], case["block"], case["d"], st["axis"].shape[0]
    theta = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = torch.stack([st["positions"][a, :n].double() for a in st["axes"]], 1) * theta
    unit = torch.polar(torch.ones_like(angle), angle)[:, None]
    # where the real and imaginary parts of pair c sit in a head's row
    c = torch.arange(half, device="cuda")
    re, im = (2 * c, 2 * c + 1) if case["interleaved"] else (c, c + half)

    def turned(x, gain):
        x = x[:n].double()
        if gain is not None:
            x = x / (x.square().sum(-1, keepdim=True) / d + st["eps"]).sqrt() * gain.double()
        z = torch.complex(x[..., re], x[..., im]) * unit
        x = x.clone()
        x[..., re], x[..., im] = z.real, z.imag
        return x

    q = st["q_out"].double()
    q[:n] = turned(st["q"], st["qw"])
    out = {"q": q}
    blk, off = torch.div(st["slots"][:n], B, rounding_mode="floor"), st["slots"][:n] % B
    for name, rows in (("k", turned(st["k"], st["kw"])), ("v", st["v"][:n].double())):
        cache = st[name + "c"]
        if case["op"] == "mrope":
            whole = cache.double()
            whole[blk, :, off] = rows
        else:
            # the values that the cache holds, and the largest of each block's positions in use
            whole = cache.view(torch.float8_e4m3fn).double()
            scales = st[name + "_scales"].cpu().numpy().astype(np.int64) - 127
            tops = rows.abs().amax(-1).cpu().numpy()
            blocks, offsets = blk.tolist(), off.tolist()
            need, begun = {}, {}
            for b, o, t in zip(blocks, offsets, tops):
                need[b] = np.maximum(need.get(b, 0.0), t)
                begun[b] = min(begun.get(b, B), o)
            for b, t in need.items():
                m, e = np.frexp(t)
                least = np.where(t > 0, np.maximum(e - 9 + (m > 0.875), -127), -127)
                after = least if begun[b] == 0 else np.maximum(least, scales[b])
                if begun[b]:
                    whole[b] *= torch.from_numpy(2.0 ** (scales[b] - after)).cuda()[:, None, None]
                scales[b] = after
            whole[blk, :, off] = rows * torch.from_numpy(2.0 ** -scales[blocks].astype(np.float64)).cuda()[..., None]
            out[name + "_scales"] = torch.from_numpy(2.0 ** scales.astype(np.float64)).cuda()
        out[name + "_cache"] = whole
    return out


def exact(case, seed):
    return (_exact_attend if case["op"] == "attend" else _exact_rope)(case, seed)
