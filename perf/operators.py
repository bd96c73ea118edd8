"""Measured cases of the operators around a paged step of new tokens.

Three operators follow one another in a serving step whose requests bring one
or a few new tokens each (decode, speculative verification, prompt chunks):

  plan   block tables, slots and positions of the step, from the requests'
         lengths and the pool's free blocks;
  rope   per-head RMS norm of q and k, rotation by position, and the write of
         k and v into the paged cache (bf16 or E4M3), in one pass;
  multi  attention of each request's few new tokens over its paged cache,
         causal or under a tree mask, bf16 or E4M3.

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
        # the smallest step: 4 requests of a test-sized engine, one token each
        dict(name="plan 4 requests", op="plan", seqs=4, spare_rows=4, block=16, max_blocks=3, median=16, longest=37,
             chunks=0, chunk=1, pad_seqs=0, pad_tokens=0),
        # one decode step of a continuous batch of 256 requests of very mixed lengths
        dict(name="plan 256 decodes", op="plan", seqs=256, spare_rows=32, block=16, max_blocks=1024, median=700,
             longest=16384, chunks=0, chunk=1, pad_seqs=0, pad_tokens=0),
        # a large mixed step of a captured graph: decodes and sixteen prompt chunks, padded batch and tokens
        dict(name="plan 1000 with chunks", op="plan", seqs=1000, spare_rows=24, block=8, max_blocks=2048, median=700,
             longest=14000, chunks=16, chunk=2003, pad_seqs=24, pad_tokens=131),
        # a few requests decoding: latency
        dict(name="rope 4 tokens", op="rope", tokens=4, pad=0, hq=32, hkv=8, d=128, rot=128, interleaved=False, norm=True,
             block=16, fp8=False, longest=4096, chunk=1),
        # a padded decode batch on a quantised cache
        dict(name="rope 250 tokens fp8", op="rope", tokens=256, pad=6, hq=32, hkv=8, d=128, rot=128, interleaved=False,
             norm=True, block=16, fp8=True, longest=32768, chunk=1),
        # prompt chunks of a model with small heads, partial interleaved rotation and no norm
        dict(name="rope 5003 tokens d64", op="rope", tokens=5003, pad=0, hq=16, hkv=2, d=64, rot=32, interleaved=True,
             norm=False, block=32, fp8=False, longest=131072, chunk=617),
        # sixteen whole prompts at once
        dict(name="rope 32048 tokens", op="rope", tokens=32048, pad=0, hq=32, hkv=8, d=128, rot=128, interleaved=False,
             norm=True, block=16, fp8=False, longest=4096, chunk=2003),
        # the smallest attention step: ragged new tokens, small heads
        dict(name="multi 4 requests d64", op="multi", seqs=4, most_new=3, hq=4, hkv=2, d=64, block=16, shortest=4,
             longest=37, tree=False, fp8=False, even=False),
        # verification of four tokens a request on the 8B-shaped batch
        dict(name="multi 64 verify 4", op="multi", seqs=64, most_new=4, hq=32, hkv=8, d=128, block=16, shortest=512,
             longest=4096, tree=False, fp8=False, even=True),
        # the same batch on a quantised cache, up to eight ragged tokens
        dict(name="multi 64 verify 8 fp8", op="multi", seqs=64, most_new=8, hq=32, hkv=8, d=128, block=16, shortest=512,
             longest=4096, tree=False, fp8=True, even=False),
        # few requests over long contexts: the keys have to be split over the whole device
        dict(name="multi 8 long verify 5", op="multi", seqs=8, most_new=5, hq=32, hkv=8, d=128, block=32, shortest=32000,
             longest=32768, tree=False, fp8=False, even=True),
        # draft trees of up to sixteen tokens
        dict(name="multi 48 trees 16", op="multi", seqs=48, most_new=16, hq=32, hkv=8, d=128, block=16, shortest=200,
             longest=6000, tree=True, fp8=False, even=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "multi"])
    block = rng.choice([8, 16, 32])
    if op == "plan":
        seqs = _log_int(rng, 1, 1000)
        longest = _log_int(rng, 30, 14000)
        chunk = _log_int(rng, 1, 2003)
        chunks = rng.randint(0, min(seqs, 16))
        return dict(op="plan", seqs=seqs, spare_rows=rng.randint(0, 40), block=block,
                    max_blocks=-(-(longest + chunk) // block) + rng.randint(0, 9),
                    median=max(1, longest // rng.randint(2, 20)), longest=longest, chunks=chunks, chunk=chunk,
                    pad_seqs=rng.randint(0, min(seqs - 1, 24)), pad_tokens=rng.randint(0, 200))
    if op == "rope":
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8])
        tokens = _log_int(rng, 1, 16000)
        return dict(op="rope", tokens=tokens, pad=rng.randint(0, tokens // 8), hq=hkv * rng.choice([1, 2, 4, 8]), hkv=hkv,
                    d=d, rot=rng.choice([16, 32, d // 2, d, d]), interleaved=rng.random() < 0.4, norm=rng.random() < 0.7,
                    block=block, fp8=rng.random() < 0.4, longest=_log_int(rng, 2000, 131072),
                    chunk=_log_int(rng, max(1, tokens // 250), 600))
    fp8 = rng.random() < 0.4
    hkv = rng.choice([1, 2, 4, 8])
    hq, most_new, longest = hkv * rng.choice([1, 2, 4, 8]), _log_int(rng, 1, 32), _log_int(rng, 40, 20000)
    most = min(200, 160000 // longest, 40_000_000 // (longest * hq * most_new))      # no dearer than the listed ones
    return dict(op="multi", seqs=_log_int(rng, 1, max(1, most)), most_new=most_new, hq=hq, hkv=hkv,
                d=128 if fp8 else rng.choice([64, 128]), block=block, shortest=max(1, longest // rng.choice([1, 4, 20])),
                longest=longest, tree=rng.random() < 0.4, fp8=fp8, even=rng.random() < 0.3)


# ---------------------------------------------------------------------------
# sizes that follow from a case alone (the seed only orders them)
# ---------------------------------------------------------------------------

def _plan_sizes(case):
    """(positions cached, new positions) of each request, in a fixed order."""
    S = case["seqs"] - case["pad_seqs"]
    u = (np.arange(S) + 0.5) / S
    # lognormal quantiles (sigma 1) around the median, by a logistic stand-in for the normal quantile
    z = np.log(u / (1 - u)) / 1.702
    lens = np.clip(np.round(case["median"] * np.exp(z)), 1, case["longest"]).astype(np.int64)
    lens -= 1                                            # a request may have nothing cached yet
    new = np.ones(S, dtype=np.int64)
    new[:min(case["chunks"], S)] = case["chunk"]
    room = case["max_blocks"] * case["block"]
    lens = np.minimum(lens, np.maximum(room - new, 0))
    return lens, np.minimum(new, room)


def _plan_tokens(case):
    return int(_plan_sizes(case)[1].sum()) + case["pad_tokens"]


def _multi_sizes(case):
    """(context length, new tokens) of each request, in a fixed order."""
    S = case["seqs"]
    u = (np.arange(S) + 0.5) / S
    ctx = np.round(case["shortest"] + u * (case["longest"] - case["shortest"])).astype(np.int64)
    m = case["most_new"]
    new = np.full(S, m) if case["even"] else 1 + (np.arange(S) * 7 + m - 1) % m
    return ctx, np.minimum(new, ctx)


def _rope_runs(case):
    """(tokens, first position) choices of the runs that make up the tokens."""
    left, runs = case["tokens"] - case["pad"], []
    while left > 0:
        runs.append(min(case["chunk"], left))
        left -= runs[-1]
    return runs


def work(case):
    if case["op"] == "plan":
        lens, new = _plan_sizes(case)
        B, S = case["block"], case["seqs"]
        held = -(-lens // B)
        total = -(-(lens + new) // B)
        taken = int((total - held).sum())
        n = 4 * 4 * S + 4 * int(held.sum()) + 4 * taken                # rows, lengths, counts, tables, free blocks
        n += 4 * S * case["max_blocks"] + 4 * (2 * S + 1) + 12 * _plan_tokens(case)
        n += 4 * taken + 4 * len(lens) + 8                             # tables and counts brought up to date
        return {"bytes": n, "flops": 0}
    if case["op"] == "rope":
        T = case["tokens"] - case["pad"]
        q, kv = case["hq"] * case["d"], 2 * case["hkv"] * case["d"]
        angles = 4 * case["rot"] * min(T, case["longest"])
        return {"bytes": T * (4 * q + 2 * kv + (1 if case["fp8"] else 2) * kv + 12) + angles,
                "flops": T * (q + kv // 2) * 8}
    ctx, new = _multi_sizes(case)
    elem = 1 if case["fp8"] else 2
    tokens = int(new.sum())
    kv = 2 * int(ctx.sum()) * case["hkv"] * case["d"] * elem
    tables = 4 * int((-(-ctx // case["block"])).sum())
    seen = int((ctx * new - new * (new - 1) // 2).sum())
    return {"bytes": kv + tables + 4 * tokens * case["hq"] * case["d"] + (8 * tokens if case["tree"] else 0),
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


def _plan_host(case, seed):
    rng = np.random.default_rng(seed)
    lens, new = _plan_sizes(case)
    order = rng.permutation(len(lens))
    lens, new = lens[order], new[order]
    S, B, MB = case["seqs"], case["block"], case["max_blocks"]
    R = S + case["spare_rows"]
    rows = rng.permutation(R)[:len(lens)]
    seq_rows = np.full(S, -1, dtype=np.int32)
    seq_rows[:len(lens)] = rows                          # the padding of a captured batch comes last
    new_lens = np.zeros(S, dtype=np.int32)
    new_lens[:len(lens)] = new
    held = -(-lens // B)
    used = int(held.sum())
    NB = used + int((-(-(lens + new) // B) - held).sum()) + 37
    ids = rng.permutation(NB).astype(np.int32)
    row_tables = np.full((R, MB), -1, dtype=np.int32)
    row_lens = np.zeros(R, dtype=np.int32)
    counts = np.zeros(R + 1, dtype=np.int32)             # blocks held per row, then the free blocks' count
    at = 0
    for r, n, h in zip(rows, lens, held):
        row_tables[r, :h] = ids[at:at + h]
        row_lens[r] = n
        counts[r] = h
        at += int(h)
    counts[R] = NB - used
    return dict(seq_rows=seq_rows, new_lens=new_lens, row_tables=row_tables, row_lens=row_lens, counts=counts,
                free_blocks=ids[used:].copy(), NB=NB, R=R, T=_plan_tokens(case))


def _prepare_plan(case, seed):
    h = _plan_host(case, seed)
    st = {k: _dev(v) for k, v in h.items() if isinstance(v, np.ndarray)}
    S, T = case["seqs"], h["T"]
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    st.update(block_tables=i32(S, case["max_blocks"]), context_lens=i32(S), query_start=i32(S + 1), positions=i32(T),
              slot_mapping=torch.zeros(T, dtype=torch.int64, device="cuda"), R=h["R"], NB=h["NB"], T=T,
              B=case["block"], counts0=st["counts"].clone())
    return st


def _prepare_rope(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    T, hq, hkv, d, B = case["tokens"], case["hq"], case["hkv"], case["d"], case["block"]
    qkv = torch.randn(T, (hq + 2 * hkv) * d, generator=g, device="cuda").mul_(1.5).to(torch.bfloat16)
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    runs = _rope_runs(case)
    pos = np.concatenate([np.arange(n) + rng.integers(0, case["longest"] - n + 1) for n in runs])
    NB = sum(-(-n // B) + 1 for n in runs) + 3
    ids, slots, at = rng.permutation(NB), [], 0
    for n in runs:                                        # each run sits in blocks of its own, from some offset on
        j = np.arange(n) + rng.integers(0, B)
        slots.append(ids[at + j // B] * B + j % B)
        at += -(-n // B) + 1
    pad = case["pad"]
    positions = np.concatenate([pos, np.full(pad, -1)]).astype(np.int32)
    slots = np.concatenate(slots + [np.full(pad, -1)]).astype(np.int64)
    half = case["rot"] // 2
    angle = torch.arange(case["longest"], dtype=torch.float64, device="cuda")[:, None] * \
        10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
    gain = lambda: 1 + 0.1 * torch.randn(d, generator=g, device="cuda")  # noqa: E731
    qw, kw = (gain(), gain()) if case["norm"] else (None, None)
    shape = (NB, hkv, B, d)
    if case["fp8"]:
        kc, vc = (torch.randn(shape, generator=g, device="cuda").mul_(60).clamp_(-448, 448).to(torch.float8_e4m3fn)
                  .view(torch.uint8) for _ in range(2))
    else:
        kc, vc = (torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    return dict(q=q, k=k, v=v, positions=_dev(positions), slots=_dev(slots), cos_sin=cos_sin, qw=qw, kw=kw, eps=1e-6,
                kc=kc, vc=vc, q_out=torch.zeros(T, hq, d, dtype=torch.bfloat16, device="cuda"), n=T - pad,
                interleaved=case["interleaved"],
                k_scale=0.0173 if case["fp8"] else None, v_scale=0.0161 if case["fp8"] else None)


def _tree_masks(new, rng):
    """Bit j of a token's word: it sees new token j (its ancestors in the draft tree, and itself)."""
    words = []
    for n in new:
        seen = []
        for i in range(n):
            up = int(rng.integers(0, i)) if i else -1
            seen.append((seen[up] if up >= 0 else 0) | (1 << i))
        words += seen
    return np.array(words, dtype=np.uint64).view(np.int64)


def _prepare_multi(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    ctx, new = _multi_sizes(case)
    order = rng.permutation(len(ctx))
    ctx, new = ctx[order], new[order]
    hq, hkv, d, B = case["hq"], case["hkv"], case["d"], case["block"]
    blocks = -(-ctx // B)
    NB, MB = int(blocks.sum()) + 5, int(blocks.max()) + 1
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
    if case["fp8"]:
        kc, vc = (torch.randn(shape, generator=g, device="cuda").mul_(60).clamp_(-448, 448).to(torch.float8_e4m3fn)
                  .view(torch.uint8) for _ in range(2))
    else:
        kc, vc = (torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(T, hq, d, generator=g, device="cuda").to(torch.bfloat16)
    return dict(q=q, kc=kc, vc=vc, tables=_dev(tables), query_start=_dev(start.astype(np.int32)),
                context_lens=_dev(ctx.astype(np.int32)), mask=_dev(_tree_masks(new, rng)) if case["tree"] else None,
                seq=_dev(seq), nth=_dev(np.arange(T) - start[seq]), new=_dev(new), most_new=case["most_new"],
                max_ctx=case["longest"], B=B, scale=1 / math.sqrt(d), hq=hq, hkv=hkv, d=d,
                out=torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda"),
                k_scale=1 / 60 if case["fp8"] else None, v_scale=1 / 60 if case["fp8"] else None)


def prepare(case, seed):
    st = {"plan": _prepare_plan, "rope": _prepare_rope, "multi": _prepare_multi}[case["op"]](case, seed)
    st["op"] = case["op"]
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _plan_outputs(st):
    return {k: st[k] for k in ("block_tables", "context_lens", "query_start", "positions", "slot_mapping", "row_tables",
                               "counts")}


def _run_plan(st):
    st["counts"].copy_(st["counts0"])                     # every pass plans the same step, from the state before it
    B, R, T = st["B"], st["R"], st["T"]
    held_rows, free_count = st["counts"][:R], st["counts"][R:]
    if own:
        from paged_kv_cache_124_gb300 import api
        api.pa_plan_step(st["block_tables"], st["context_lens"], st["query_start"], st["positions"], st["slot_mapping"],
                         st["seq_rows"], st["new_lens"], st["row_lens"], st["row_tables"], held_rows, st["free_blocks"],
                         free_count, B, st["NB"])
        return _plan_outputs(st)
    real = st["seq_rows"] >= 0
    r = st["seq_rows"].clamp(min=0).long()
    cached = torch.where(real, st["row_lens"][r], 0)
    new = torch.where(real, st["new_lens"], 0)
    held = torch.where(real, held_rows[r], 0)
    need = torch.where(real, ((cached + new + B - 1) // B - held).clamp(min=0), 0)
    ends = need.cumsum(0)
    fits = ends[-1:] <= free_count                        # all or nothing
    need, new = need * fits, new * fits
    ctx = cached + new
    j = torch.arange(st["row_tables"].shape[1], device="cuda")
    nth = (ends - need - held)[:, None] + j               # which of the step's blocks entry j takes
    fresh = (j >= held[:, None]) & (j < (held + need)[:, None])
    old = st["row_tables"][r]
    take = (free_count - 1 - nth).clamp(0, st["free_blocks"].shape[0] - 1).long()
    entries = torch.where(fresh, st["free_blocks"][take], old)
    st["row_tables"].index_put_((r,), torch.where(fresh, entries - old, 0), accumulate=True)
    held_rows.index_put_((r,), need.int(), accumulate=True)
    free_count -= need.sum().int()
    st["block_tables"].copy_(torch.where(j < ((ctx + B - 1) // B)[:, None], entries, -1))
    st["context_lens"].copy_(ctx)
    st["query_start"][1:] = new.cumsum(0)
    t = torch.arange(T, device="cuda")
    i = torch.searchsorted(st["query_start"][1:], t.int(), right=True).clamp(max=len(r) - 1)
    pos = ctx[i] - new[i] + t - st["query_start"][i]
    inside = t < st["query_start"][-1]
    slot = st["block_tables"][i, (pos // B).clamp(0, len(j) - 1)].long() * B + pos % B
    st["positions"].copy_(torch.where(inside, pos, -1))
    st["slot_mapping"].copy_(torch.where(inside, slot, -1))
    return _plan_outputs(st)


def _rope_outputs(st):
    kc, vc = st["kc"], st["vc"]
    if st["k_scale"] is not None:
        kc, vc = kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn)
    return {"q": st["q_out"], "k_cache": kc, "v_cache": vc}


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


def _run_rope(st):
    if own:
        from paged_kv_cache_124_gb300 import api
        api.pa_qk_norm_rope_cache(st["q_out"], st["kc"], st["vc"], st["q"], st["k"], st["v"], st["positions"],
                                  st["slots"], st["cos_sin"], q_weight=st["qw"], k_weight=st["kw"], eps=st["eps"],
                                  interleaved=st["interleaved"], k_scale=st["k_scale"], v_scale=st["v_scale"])
        return _rope_outputs(st)
    n, B = st["n"], st["kc"].shape[2]
    cos, sin = st["cos_sin"][st["positions"][:n].long()].chunk(2, -1)
    cos, sin = cos[:, None], sin[:, None]
    q = _plain_norm_rope(st["q"][:n], st["qw"], st["eps"], cos, sin, st["interleaved"])
    k = _plain_norm_rope(st["k"][:n], st["kw"], st["eps"], cos, sin, st["interleaved"])
    v = st["v"][:n].float()
    if st["k_scale"] is None:
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    else:
        k, v = ((x / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                for x, s in ((k, st["k_scale"]), (v, st["v_scale"])))
    st["q_out"][:n] = q.to(torch.bfloat16)
    blk, off = st["slots"][:n] // B, st["slots"][:n] % B
    st["kc"][blk, :, off] = k
    st["vc"][blk, :, off] = v
    return _rope_outputs(st)


def _gathered(cache, tables, scale):
    """A cache's positions in order, [S, Hkv, positions, D] in 32 bits."""
    x = cache[tables.clamp(min=0).long()]
    x = x.float() if scale is None else x.view(torch.float8_e4m3fn).float() * scale
    S, MB, H, B, D = x.shape
    return x.transpose(1, 2).reshape(S, H, MB * B, D)


def _run_multi(st):
    if own:
        from paged_kv_cache_124_gb300 import api
        if "workspace" not in st:
            st["workspace"] = api.decode_multi_workspace(st["most_new"], st["hq"], st["hkv"], st["d"])
        api.pa_decode_multi(st["out"], st["q"], st["kc"], st["vc"], st["tables"], st["query_start"], st["context_lens"],
                            st["most_new"], st["B"], st["scale"], st["hq"], st["hkv"], st["d"], st["max_ctx"],
                            tree_mask=st["mask"], workspace=st["workspace"], k_scale=st["k_scale"],
                            v_scale=st["v_scale"])
        return st["out"]
    S, m, G = st["tables"].shape[0], st["most_new"], st["hq"] // st["hkv"]
    K = _gathered(st["kc"], st["tables"], st["k_scale"])
    V = _gathered(st["vc"], st["tables"], st["v_scale"])
    i = torch.arange(m, device="cuda")
    at = (st["query_start"][:-1, None] + i).clamp(max=st["q"].shape[0] - 1).long()    # token i of each request
    q = st["q"][at].float().unflatten(2, (st["hkv"], G)).permute(0, 2, 1, 3, 4).reshape(S, st["hkv"], m * G, -1)
    j = torch.arange(K.shape[2], device="cuda")
    first = (st["context_lens"] - st["new"])[:, None, None]        # position of a request's first new token
    if st["mask"] is None:
        seen = j <= first + i[:, None]
    else:
        bit = (j - first).clamp(0, 63)
        seen = (j < first) | ((j - first < st["new"][:, None, None]) & ((st["mask"][at][:, :, None] >> bit) & 1 == 1))
    s = (q @ K.transpose(-1, -2)).unflatten(2, (m, G)) * st["scale"]
    s = s.masked_fill(~seen[:, None, :, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = (s - torch.where(top > -math.inf, top, 0)).exp()
    total = p.sum(-1, keepdim=True)
    o = p.flatten(2, 3) @ V
    o = o.unflatten(2, (m, G)) / torch.where(total > 0, total, 1)
    o = o.permute(0, 2, 1, 3, 4).flatten(2, 3)                     # [S, m, Hq, D]
    st["out"].copy_(o[st["seq"], st["nth"]])
    return st["out"]


def run(state):
    return {"plan": _run_plan, "rope": _run_rope, "multi": _run_multi}[state["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_plan(case, seed):
    h = _plan_host(case, seed)
    B, MB, T = case["block"], case["max_blocks"], h["T"]
    stack = h["free_blocks"].tolist()
    tables = np.full((case["seqs"], MB), -1, dtype=np.int32)
    ctxs, starts, positions, slots = [], [0], [], []
    for i, (r, n) in enumerate(zip(h["seq_rows"].tolist(), h["new_lens"].tolist())):
        cached = int(h["row_lens"][r]) if r >= 0 else 0
        for p in range(cached, cached + n):
            if p // B >= h["counts"][r]:
                h["row_tables"][r, p // B] = stack.pop()
                h["counts"][r] += 1
            positions.append(p)
            slots.append(int(h["row_tables"][r, p // B]) * B + p % B)
        ctxs.append(cached + n)
        starts.append(starts[-1] + n)
        nb = -(-ctxs[-1] // B)
        if nb:
            tables[i, :nb] = h["row_tables"][r, :nb]
    h["counts"][-1] = len(stack)
    pad = T - len(positions)
    return dict(block_tables=tables, context_lens=np.array(ctxs, np.int32), query_start=np.array(starts, np.int32),
                positions=np.array(positions + [-1] * pad, np.int32), slot_mapping=np.array(slots + [-1] * pad, np.int64),
                row_tables=h["row_tables"], counts=h["counts"])


def _exact_rope(case, seed):
    st = _prepare_rope(case, seed)
    n, B, d, half = st["n"], case["block"], case["d"], case["rot"] // 2
    theta = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    unit = torch.polar(torch.ones(n, half, dtype=torch.float64, device="cuda"),
                       st["positions"][:n].double()[:, None] * theta)[:, None]
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
    for name, cache, rows, s in (("k_cache", st["kc"], turned(st["k"], st["kw"]), st["k_scale"]),
                                 ("v_cache", st["vc"], st["v"][:n].double(), st["v_scale"])):
        whole = cache.view(torch.float8_e4m3fn).double() if s is not None else cache.double()
        whole[blk, :, off] = rows if s is None else (rows / s).clamp(-448, 448)
        out[name] = whole
    return out


def _exact_multi(case, seed):
    st = _prepare_multi(case, seed)
    B, G, hkv, d = st["B"], st["hq"] // st["hkv"], st["hkv"], st["d"]
    start, ctxs = st["query_start"].tolist(), st["context_lens"].tolist()
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for s, C in enumerate(ctxs):
        lo, hi = start[s], start[s + 1]
        n = hi - lo
        ids = st["tables"][s, :-(-C // B)].long()

        def rows(cache, scale):
            x = cache[ids] if scale is None else cache[ids].view(torch.float8_e4m3fn)
            x = x.double() if scale is None else x.double() * scale
            return x.permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, :C]

        K, V = rows(st["kc"], st["k_scale"]), rows(st["vc"], st["v_scale"])
        see = torch.ones(n, C, dtype=torch.bool, device="cuda")
        if st["mask"] is None:
            see[:, C - n:] = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        else:
            words = [w & (2 ** 64 - 1) for w in st["mask"][lo:hi].tolist()]
            see[:, C - n:] = torch.tensor([[(w >> b) & 1 == 1 for b in range(n)] for w in words], device="cuda")
        q = st["q"][lo:hi].double().view(n, hkv, G, d)
        logits = torch.einsum("nhgd,hcd->hgnc", q, K) * st["scale"]
        logits = torch.where(see, logits, torch.full_like(logits, -math.inf))
        out[lo:hi] = torch.einsum("hgnc,hcd->nhgd", torch.softmax(logits, -1), V).reshape(n, st["hq"], d)
    return out


def exact(case, seed):
    return {"plan": _exact_plan, "rope": _exact_rope, "multi": _exact_multi}[case["op"]](case, seed)
