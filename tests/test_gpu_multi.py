"""pa_decode_multi and pa_decode_multi_fp8 against the float64 oracle, at the
sizes, masks and lengths where they can go wrong."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import quant as Q
from _gpu_util import from_bits, out_to_f64, to_bits

pytestmark = pytest.mark.gpu

api = pytest.importorskip("paged_kv_cache_124_gb300.api")
from paged_kv_cache_124_gb300 import inputs as I  # noqa: E402

K_SCALE, V_SCALE = 0.02, 0.03


def _problem(seed, Hq, Hkv, D, B, ctxs, news, fp8=False, gap=0):
    """Filled slots up to each context, NaN in every other; `gap` rows of q
    and out before, between and behind the sequences' rows belong to none."""
    rng = np.random.default_rng(seed)
    nblk = [-(-c // B) for c in ctxs]
    NB, MB = sum(nblk) + 4, max(nblk + [1]) + 1
    ids = rng.permutation(NB).astype(np.int32)
    tables, at = np.full((len(ctxs), MB), -1, dtype=np.int32), 0
    for s, n in enumerate(nblk):
        tables[s, :n] = ids[at:at + n]
        at += n
    if fp8:
        draw = lambda: Q.quantize(np.clip(rng.standard_normal((NB, Hkv, B, D)), -4, 4), 0.02)  # noqa: E731
    else:
        draw = lambda: to_bits(I.bf16_normal((NB, Hkv, B, D), int(rng.integers(1 << 30))))  # noqa: E731
    nan = 0x7F if fp8 else 0x7FC0
    kc, vc = draw(), draw()
    filled = np.zeros((NB, B), dtype=bool)
    for s, c in enumerate(ctxs):
        for j in range(nblk[s]):
            filled[tables[s, j], :min(B, c - j * B)] = True
    for c in (kc, vc):
        blk, off = np.where(~filled)
        c[blk, :, off] = nan
    start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32) + gap
    T = int(start[-1]) + gap
    q = I.bf16_normal((T, Hq, D), seed + 1)
    return q, kc, vc, tables, start, np.array(ctxs, dtype=np.int32)


def _run(p, Hq, Hkv, D, B, most, out_dtype=torch.float32, mask=None, fp8=False, scale=None, max_ctx=None, ws=None,
         status=None, stream=None):
    q, kc, vc, tables, start, ctx = p
    dev = "cuda"
    out = torch.full(q.shape, float("nan"), dtype=out_dtype, device=dev)
    put = (lambda c: torch.from_numpy(c).to(dev)) if fp8 else (lambda c: from_bits(c))
    m = None if mask is None else torch.from_numpy(np.array(mask, dtype=np.uint64).view(np.int64)).to(dev)
    api.pa_decode_multi(out, q.to(dev), put(kc), put(vc), torch.from_numpy(tables).to(dev),
                        torch.from_numpy(start).to(dev), torch.from_numpy(ctx).to(dev), most, B,
                        1 / math.sqrt(D) if scale is None else scale, Hq, Hkv, D,
                        int(ctx.max()) if max_ctx is None else max_ctx, tree_mask=m,
                        workspace=api.decode_multi_workspace(most, Hq, Hkv, D) if ws is None else ws, status=status,
                        k_scale=K_SCALE if fp8 else None, v_scale=V_SCALE if fp8 else None)
    return out


def _check(p, out, Hq, Hkv, D, B, mask=None, fp8=False, scale=None, skip=()):
    """|out - ref| within what the roundings inside allow: a weight is off by
    a relative 2 (E + 128 * 2^-24) * (|q| . |k|) |scale| + W, E and W the
    operand roundings (bf16: q exact, weights in two terms, W 2^-16; E4M3: q
    and weights to f16, 2^-11 each), doubled as the normaliser moves too; an
    output by that times sum a |v|; and half a step of the output's type.
    E4M3, besides: more than 16 rows take weights as E5M2 terms, scaled so that
    a row's largest is 2^12 at least (2^15 with a headroom of 2^3) and cut off
    at E5M2's smallest step, 2^-16: a weight may lose 2^-28 of the largest,
    and, the normaliser being at least the largest, an output 2^-28 sum |v|.
    (f16, up to 16 rows: the largest is 2^7 at least, half a step 2^-25:
    2^-32.)"""
    q, kc, vc, tables, start, ctx = p
    scale = 1 / math.sqrt(D) if scale is None else scale
    kd, vd = (Q.dequantize(kc, K_SCALE), Q.dequantize(vc, V_SCALE)) if fp8 else (kc, vc)
    want = A.paged_multi(to_bits(q), kd, vd, tables, start, ctx, scale, B, mask)
    f64 = (lambda c: c) if fp8 else A.bf16_to_f64
    weight = A.paged_multi(to_bits(q), f64(kd), np.abs(f64(vd)), tables, start, ctx, scale, B, mask)
    E, W = (2.0 ** -11, 2.0 ** -11) if fp8 else (0.0, 2.0 ** -16)
    got = out_to_f64(out)
    qa = np.abs(A.bf16_to_f64(to_bits(q)))
    covered = np.zeros(q.shape[0], dtype=bool)
    for s in range(len(ctx)):
        if s in skip:
            continue
        K, V = A.gather_kv(np.abs(f64(kd)), np.abs(f64(vd)), tables[s], int(ctx[s]), B)
        for r in range(start[s], start[s + 1]):
            covered[r] = True
            for g in range(Hq):
                size = (K[g // (Hq // Hkv)] @ qa[r, g]).max() * abs(scale)
                tol = (2 * (E + 128 * 2.0 ** -24) * size + W + 2.0 ** -18) * weight[r, g] * 2
                if fp8:
                    tol = tol + 2.0 ** -28 * V[g // (Hq // Hkv)].sum(0)
                if out.dtype == torch.bfloat16:
                    tol = tol + 2.0 ** -8 * np.abs(want[r, g])
                assert (np.abs(got[r, g] - want[r, g]) <= tol).all(), (s, r, g, np.abs(got[r, g] - want[r, g]).max())
    assert np.isnan(got[~covered]).all()                       # rows of no sequence are left as they were


def _trees(news, rng):
    words = []
    for n in news:
        seen = []
        for i in range(n):
            up = int(rng.integers(-1, i)) if i else -1
            seen.append((seen[up] if up >= 0 else 0) | 1 << i)
        words += seen
    return words


CASES = [
    # Hq, Hkv, D, B, contexts, new tokens
    (4, 2, 64, 16, [2, 16, 17, 38], [1, 2, 3, 1]),
    (32, 8, 128, 16, [1, 65, 300, 1000], [1, 4, 4, 2]),            # 16 rows: two column tiles
    (8, 8, 128, 8, [8, 9, 70, 513], [8, 1, 5, 7]),                 # G = 1, 8-position blocks
    (8, 4, 64, 32, [31, 64, 200], [16, 3, 9]),                     # 32 rows
    (32, 2, 128, 16, [40, 129], [3, 9]),                           # G = 16: 144 rows, five row tiles
    (16, 2, 64, 8, [61, 12], [20, 12]),                            # a whole prompt of 12
    (2, 1, 128, 32, [2500], [2]),                                  # one head: the keys over many blocks
]


@pytest.mark.parametrize("Hq,Hkv,D,B,ctxs,news", CASES)
@pytest.mark.parametrize("kind", ["causal", "tree"])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_multi_equals_the_oracle(Hq, Hkv, D, B, ctxs, news, kind, out_dtype):
    p = _problem(Hq + D + B, Hq, Hkv, D, B, ctxs, news, gap=2)
    rng = np.random.default_rng(1)
    mask = None
    if kind == "tree":
        mask = [0, 0] + _trees(news, rng) + [0, 0]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _run(p, Hq, Hkv, D, B, max(news), out_dtype, mask, status=st)
    assert st.item() == 0
    _check(p, out, Hq, Hkv, D, B, mask)


@pytest.mark.parametrize("Hq,Hkv,D,B,ctxs,news", [c for c in CASES if c[2] == 128])
@pytest.mark.parametrize("kind", ["causal", "tree"])
def test_multi_fp8_equals_the_oracle(Hq, Hkv, D, B, ctxs, news, kind):
    p = _problem(Hq + B, Hq, Hkv, D, B, ctxs, news, fp8=True, gap=1)
    mask = [0] + _trees(news, np.random.default_rng(2)) + [0] if kind == "tree" else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _run(p, Hq, Hkv, D, B, max(news), mask=mask, fp8=True, status=st)
    assert st.item() == 0
    _check(p, out, Hq, Hkv, D, B, mask, fp8=True)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_one_token_is_the_decode(fp8):
    """n = 1 for every sequence: pa_decode's operation."""
    Hq, Hkv, D, B, ctxs = 32, 8, 128, 16, [1, 30, 700, 2100]
    p = _problem(3, Hq, Hkv, D, B, ctxs, [1] * 4, fp8=fp8)
    _check(p, _run(p, Hq, Hkv, D, B, 1, fp8=fp8), Hq, Hkv, D, B, fp8=fp8)


@pytest.mark.parametrize("D", [64, 128])
def test_sixty_four_tokens_and_whole_prompts(D):
    Hq, Hkv, B, ctxs, news = 4, 1, 16, [64, 100, 63], [64, 64, 63]
    p = _problem(4, Hq, Hkv, D, B, ctxs, news)
    words = _trees(news, np.random.default_rng(3))
    words[63] |= 1 << 63
    _check(p, _run(p, Hq, Hkv, D, B, 64, mask=words), Hq, Hkv, D, B, words)
    _check(p, _run(p, Hq, Hkv, D, B, 64), Hq, Hkv, D, B)


def test_chunks_past_sixty_four_tokens_are_causal():
    Hq, Hkv, D, B, ctxs, news = 4, 2, 64, 16, [150, 90], [100, 70]
    p = _problem(5, Hq, Hkv, D, B, ctxs, news)
    _check(p, _run(p, Hq, Hkv, D, B, 100), Hq, Hkv, D, B)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_rows_that_see_nothing_are_zero(fp8):
    """Nothing cached and an empty word: zeros; bits from n on say nothing; a
    row that sees only the last of many new tokens."""
    Hq, Hkv, D, B, ctxs, news = 8, 2, 128, 16, [5, 40, 33], [5, 40, 3]
    p = _problem(6, Hq, Hkv, D, B, ctxs, news, fp8=fp8)
    words = [0, 1, ~0 << 5 & (2 ** 64 - 1), 4, 31] + [0] * 39 + [1 << 39] + [0, 0, 0]
    words[5] = 1 << 39
    out = _run(p, Hq, Hkv, D, B, 40, mask=words, fp8=fp8)
    _check(p, out, Hq, Hkv, D, B, words, fp8=fp8)
    assert (out[0] == 0).all() and (out[2] == 0).all() and (out[6] == 0).all() and (out[5] != 0).any()
    assert (out[45:] != 0).any()                             # the context before the new tokens is always seen


def test_scores_of_every_size():
    """Maxima that grow along the sequence by more than the kernel lets pass
    without a rescale, fall, and differ between rows; a scale of zero."""
    Hq, Hkv, D, B, C, n = 4, 1, 128, 16, 900, 4
    q, kc, vc, tables, start, ctx = _problem(7, Hq, Hkv, D, B, [C], [n])
    k = A.bf16_to_f64(kc)
    for j in range(C):
        k[tables[0, j // B], :, j % B] *= 4.0 * (1 + math.sin(j / 70.0)) * (1 if j < 600 else 0.01)
    kc = to_bits(torch.from_numpy(np.nan_to_num(k, nan=0.0)).to(torch.bfloat16))
    p = (q, kc, vc, tables, start, ctx)
    _check(p, _run(p, Hq, Hkv, D, B, n), Hq, Hkv, D, B)
    _check(p, _run(p, Hq, Hkv, D, B, n, scale=0.0), Hq, Hkv, D, B, scale=0.0)
    _check(p, _run(p, Hq, Hkv, D, B, n, scale=-0.05), Hq, Hkv, D, B, scale=-0.05)


def test_a_nan_key_makes_its_rows_nan_and_no_other():
    Hq, Hkv, D, B = 8, 2, 64, 16
    p = _problem(8, Hq, Hkv, D, B, [300, 40], [3, 2])
    q, kc, vc, tables, start, ctx = p
    kc[tables[0, 18], 1, 10, 5] = 0x7FC0                     # position 298: the second of the three new tokens
    out = out_to_f64(_run(p, Hq, Hkv, D, B, 3))
    assert np.isnan(out[1:3, 4:]).all() and np.isfinite(out[0]).all() and np.isfinite(out[1:3, :4]).all()
    assert np.isfinite(out[3:]).all()


def test_many_ragged_sequences_and_sequences_that_bring_nothing():
    """More sequences than a block has threads, lengths from one up, some of
    them without new tokens, all in one launch over all SMs."""
    Hq, Hkv, D, B = 4, 2, 64, 8
    rng = np.random.default_rng(9)
    news = [int(x) for x in rng.integers(0, 4, 300)]
    ctxs = [int(max(1, n + rng.integers(0, 90))) for n in news]
    p = _problem(9, Hq, Hkv, D, B, ctxs, news)
    _check(p, _run(p, Hq, Hkv, D, B, 3, torch.bfloat16), Hq, Hkv, D, B)


def test_the_same_call_twice_gives_the_same_bits_and_any_workspace_serves():
    Hq, Hkv, D, B, ctxs, news = 32, 8, 128, 16, [4000, 10, 1500], [4, 4, 2]
    p = _problem(10, Hq, Hkv, D, B, ctxs, news)
    a = _run(p, Hq, Hkv, D, B, 4)
    ws = api.decode_multi_workspace(4, Hq, Hkv, D)
    ws.fill_(0xFF)
    b = _run(p, Hq, Hkv, D, B, 4, ws=ws)
    assert torch.equal(a.view(torch.int32), b.view(torch.int32))
    with pytest.raises(api.PAError) as e:
        _run(p, Hq, Hkv, D, B, 4, ws=ws[:-256])
    assert e.value.status == api.PA_ERR_WORKSPACE


def test_bad_metadata_is_flagged_and_skipped():
    Hq, Hkv, D, B, ctxs, news = 8, 2, 64, 16, [50, 30, 20, 40], [2, 3, 2, 2]
    q, kc, vc, tables, start, ctx = _problem(11, Hq, Hkv, D, B, ctxs, news)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad, most, skip in ((dict(ctx=[50, 2, 20, 40]), 3, {1}), (dict(), 2, {1}),
                            (dict(start=[0, 2, 5, 7, 10]), 3, {3})):
        p = (q, kc, vc, tables, np.array(bad.get("start", start), dtype=np.int32),
             np.array(bad.get("ctx", ctx), dtype=np.int32))
        st.zero_()
        out = _run(p, Hq, Hkv, D, B, most, status=st)
        assert st.item() == api.PA_DEV_BAD_CONTEXT
        good = (q, kc, vc, tables, start, ctx)
        _check(good, out, Hq, Hkv, D, B, skip=skip)
    # a table entry outside the pool is flagged; the other sequences are right
    t = tables.copy()
    t[2, 0] = 10 ** 6
    st.zero_()
    out = _run((q, kc, vc, t, start, ctx), Hq, Hkv, D, B, 3, status=st)
    assert st.item() == api.PA_DEV_BAD_BLOCK_ID
    out[start[2]:start[3]] = float("nan")
    _check((q, kc, vc, tables, start, ctx), out, Hq, Hkv, D, B, skip={2})


def test_on_a_stream_of_its_own():
    Hq, Hkv, D, B, ctxs, news = 8, 2, 128, 16, [500, 70], [4, 3]
    p = _problem(12, Hq, Hkv, D, B, ctxs, news)
    a = _run(p, Hq, Hkv, D, B, 4)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        b = _run(p, Hq, Hkv, D, B, 4)
    side.synchronize()
    assert torch.equal(a.view(torch.int32), b.view(torch.int32))


@pytest.mark.parametrize("i", range(24))
def test_random_configurations(i):
    rng = np.random.default_rng(100 + i)
    fp8 = bool(rng.random() < 0.4)
    D = 128 if fp8 else int(rng.choice([64, 128]))
    B, Hkv, G = int(rng.choice([8, 16, 32])), int(rng.choice([1, 2, 3, 4])), int(rng.choice([1, 2, 4, 8, 16]))
    n_seqs, most = int(rng.integers(1, 7)), int(rng.choice([1, 2, 3, 4, 7, 12, 20]))
    news = [int(x) for x in rng.integers(0, most + 1, n_seqs)]
    news[0] = most
    ctxs = [int(n + rng.choice([0, 1, 15, 16, 17, 47, 48, 64, 200, 700])) for n in news]
    ctxs = [max(1, c) for c in ctxs]
    p = _problem(200 + i, G * Hkv, Hkv, D, B, ctxs, news, fp8=fp8, gap=int(rng.integers(0, 3)))
    mask = None
    if rng.random() < 0.5:
        gap = int(p[4][0])
        mask = [0] * gap + _trees(news, rng) + [0] * gap
    dt = torch.float32 if rng.random() < 0.5 else torch.bfloat16
    _check(p, _run(p, G * Hkv, Hkv, D, B, most, dt, mask, fp8), G * Hkv, Hkv, D, B, mask, fp8)


# More than 16 rows a KV head: units of 64 rows, or 128 for bf16 caches.
WIDE = [
    (32, 8, 128, 16, [64, 65, 128, 129, 700, 16], [5, 16, 16, 9, 12, 16]),   # 64 rows; contexts of half a tile
    (16, 2, 64, 8, [64, 63, 200, 8, 193], [8, 5, 6, 8, 1]),                  # 64 rows, 8-position blocks
    (16, 1, 128, 32, [30, 128, 257, 520, 8], [5, 8, 7, 8, 8]),               # 128 rows
    (16, 2, 64, 16, [40, 300, 64], [12, 16, 16]),                            # 128 rows, d_head 64
    (8, 1, 128, 16, [9000, 33], [8, 3]),                                     # one head over many blocks
    (4, 1, 128, 8, [300, 260], [64, 40]),                                    # tree words over tile boundaries
    (1, 1, 128, 16, [100, 90, 64], [40, 17, 64]),                            # G = 1
]


@pytest.mark.parametrize("Hq,Hkv,D,B,ctxs,news", WIDE)
@pytest.mark.parametrize("kind", ["causal", "tree"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_units_of_many_rows_equal_the_oracle(Hq, Hkv, D, B, ctxs, news, kind, fp8):
    if fp8 and D != 128:
        pytest.skip("E4M3 caches have d_head 128")
    p = _problem(Hq + D + B, Hq, Hkv, D, B, ctxs, news, fp8=fp8, gap=3)
    mask = [0] * 3 + _trees(news, np.random.default_rng(4)) + [0] * 3 if kind == "tree" else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _run(p, Hq, Hkv, D, B, max(news), torch.bfloat16, mask, fp8, status=st)
    assert st.item() == 0
    _check(p, out, Hq, Hkv, D, B, mask, fp8)


@pytest.mark.parametrize("n", [4, 16, 32])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_growing_scores_and_scales_of_either_sign(n, fp8):
    """Maxima that rise by far more than a raise's threshold, again and again,
    and fall; scales of zero and below."""
    Hq, Hkv, D, B, C = 4, 1, 128, 16, 900
    q, kc, vc, tables, start, ctx = _problem(13, Hq, Hkv, D, B, [C], [n], fp8=fp8)
    k = np.nan_to_num(Q.dequantize(kc, 0.02) if fp8 else A.bf16_to_f64(kc), nan=0.0)
    for j in range(C):
        k[tables[0, j // B], :, j % B] *= 4.0 * (1 + math.sin(j / 70.0)) * (1 if j < 600 else 0.01)
    kc = Q.quantize(np.clip(k, -8.5, 8.5), K_SCALE) if fp8 else to_bits(torch.from_numpy(k).to(torch.bfloat16))
    p = (q, kc, vc, tables, start, ctx)
    for scale in (1 / math.sqrt(D), 0.0, -0.05):
        _check(p, _run(p, Hq, Hkv, D, B, n, scale=scale, fp8=fp8), Hq, Hkv, D, B, scale=scale, fp8=fp8)


# (new tokens, G, fp8): units of 16, 64 and 128 rows
UNITS = [(4, 4, False), (4, 4, True), (9, 4, False), (9, 4, True), (20, 4, False)]


@pytest.mark.parametrize("n,G,fp8", UNITS)
@pytest.mark.parametrize("kind", ["causal", "tree"])
@pytest.mark.parametrize("C", [40, 70, 3000])
def test_values_that_are_not_finite_reach_the_rows_that_see_them_alone(n, G, fp8, kind, C):
    Hkv, D, B = 2, 128, 16
    p = _problem(14, G * Hkv, Hkv, D, B, [C, 200], [n, 3], fp8=fp8)
    q, kc, vc, tables, start, ctx = p
    words = _trees([n, 3], np.random.default_rng(5)) if kind == "tree" else None
    bad = [0x7F, 0xFF, 0x7F] if fp8 else [0x7F80, 0xFF80, 0x7FC0]
    clean = vc.copy()
    for i, (j, d) in enumerate(((1, 5), (n // 2, 64), (n // 2, 5), (n - 1, 127), (n - 1, 5))):
        at = tables[0, (C - n + j) // B], i % Hkv, (C - n + j) % B, d
        vc[at], clean[at] = bad[i % 3], 0
    at = tables[0, (C - n + 2) // B], 0, (C - n + 2) % B, 7       # and a key that is not
    kc[at] = bad[2]
    f64 = (lambda c: Q.dequantize(c, V_SCALE)) if fp8 else A.bf16_to_f64
    scale = 1 / math.sqrt(D)
    args = (tables, start, ctx, scale, B, words)
    k64 = Q.dequantize(kc, K_SCALE) if fp8 else A.bf16_to_f64(kc)
    with np.errstate(invalid="ignore"):
        want = A.paged_multi(A.bf16_to_f64(to_bits(q)), k64, f64(vc), *args)
        out = _run(p, G * Hkv, Hkv, D, B, n, mask=words, fp8=fp8)
        got = out_to_f64(out)
        odd = ~np.isfinite(want)
        assert odd.any() and not odd.all()
        assert (np.isnan(got[odd]) == np.isnan(want[odd])).all()
        inf = odd & ~np.isnan(want)
        assert (got[inf] == want[inf]).all()
    # everything else is what finite values give
    k_clean = kc.copy()
    k_clean[at] = 0
    rest = out.clone()
    fine = A.paged_multi(A.bf16_to_f64(to_bits(q)), Q.dequantize(k_clean, K_SCALE) if fp8 else A.bf16_to_f64(k_clean),
                         f64(clean), *args)
    rest[torch.from_numpy(odd).cuda()] = torch.from_numpy(fine[odd]).float().cuda()
    _check((q, k_clean, clean, tables, start, ctx), rest, G * Hkv, Hkv, D, B, words, fp8)


@pytest.mark.parametrize("n,G,fp8", UNITS)
def test_bad_blocks_and_lengths_of_one_sequence_leave_the_others(n, G, fp8):
    Hkv, D, B = 2, 128, 16
    ctxs, news = [50, 300, 150, 40], [2, n, n, 3]
    p = _problem(15, G * Hkv, Hkv, D, B, ctxs, news, fp8=fp8)
    q, kc, vc, tables, start, ctx = p
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for entry in (-1, 10 ** 6):
        t = tables.copy()
        t[2, 3] = entry
        st.zero_()
        out = _run((q, kc, vc, t, start, ctx), G * Hkv, Hkv, D, B, n, fp8=fp8, status=st)
        assert st.item() == api.PA_DEV_BAD_BLOCK_ID
        out[start[2]:start[3]] = float("nan")
        _check(p, out, G * Hkv, Hkv, D, B, fp8=fp8, skip={2})
    for bad in (np.array([50, n - 1, 150, 40]), np.array([50, -7, 150, 40])):
        st.zero_()
        out = _run((q, kc, vc, tables, start, bad.astype(np.int32)), G * Hkv, Hkv, D, B, n, fp8=fp8, status=st)
        assert st.item() == api.PA_DEV_BAD_CONTEXT
        assert torch.isnan(out[start[1]:start[2]]).all()          # not computed, left as it was
        _check(p, out, G * Hkv, Hkv, D, B, fp8=fp8, skip={1})
    # a context above max_context_len is cut there
    st.zero_()
    out = _run(p, G * Hkv, Hkv, D, B, n, fp8=fp8, status=st, max_ctx=150)
    assert st.item() == api.PA_DEV_BAD_CONTEXT
    _check((q, kc, vc, tables, start, np.minimum(ctx, 150).astype(np.int32)), out, G * Hkv, Hkv, D, B, fp8=fp8)


@pytest.mark.parametrize("n,G,fp8", UNITS)
def test_no_new_tokens_and_empty_batches(n, G, fp8):
    Hkv, D, B = 2, 128, 16
    p = _problem(16, G * Hkv, Hkv, D, B, [40, 70], [0, 0], fp8=fp8, gap=2)
    assert torch.isnan(_run(p, G * Hkv, Hkv, D, B, n, fp8=fp8)).all()
    q, kc, vc, tables, start, ctx = p
    zero = (q, kc, vc, tables, np.zeros(3, dtype=np.int32), np.zeros(2, dtype=np.int32))
    assert torch.isnan(_run(zero, G * Hkv, Hkv, D, B, n, fp8=fp8, max_ctx=0)).all()


@pytest.mark.parametrize("n,G,fp8", UNITS)
def test_captured_calls_that_share_a_workspace_and_calls_on_two_streams(n, G, fp8):
    Hkv, D, B = 2, 128, 16
    Hq = G * Hkv
    probs = [_problem(17 + x, Hq, Hkv, D, B, ctxs, news, fp8=fp8)
             for x, (ctxs, news) in enumerate((([1500, 40, 700], [n, 3, n]), ([90, 2500], [n, 2])))]
    want = [_run(p, Hq, Hkv, D, B, n, fp8=fp8) for p in probs]
    put = (lambda c: torch.from_numpy(c).cuda()) if fp8 else from_bits

    def call(p, ws):
        q, kc, vc, tables, start, ctx = p
        a = [q.cuda(), put(kc), put(vc)] + [torch.from_numpy(x).cuda() for x in (tables, start, ctx)]
        out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
        return out, lambda: api.pa_decode_multi(out, *a, n, B, 1 / math.sqrt(D), Hq, Hkv, D, int(ctx.max()), workspace=ws,
                                                k_scale=K_SCALE if fp8 else None, v_scale=V_SCALE if fp8 else None)

    shared = api.decode_multi_workspace(n, Hq, Hkv, D)
    calls = [call(p, shared) for p in probs]
    graphs = []
    for _, run in calls:
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    for _ in range(3):
        for out, _ in calls:
            out.fill_(float("nan"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (out, _), w in zip(calls, want):
            assert torch.equal(out.view(torch.int32), w.view(torch.int32))
    # at once, each with a workspace of its own
    calls = [call(p, api.decode_multi_workspace(n, Hq, Hkv, D)) for p in probs]
    streams = [torch.cuda.Stream() for _ in probs]
    torch.cuda.synchronize()
    for _ in range(20):
        for (_, run), s in zip(calls, streams):
            with torch.cuda.stream(s):
                run()
    torch.cuda.synchronize()
    for (out, _), w in zip(calls, want):
        assert torch.equal(out.view(torch.int32), w.view(torch.int32))


@pytest.mark.parametrize("n,G,fp8", UNITS)
def test_long_contexts_in_the_last_blocks_of_a_large_cache(n, G, fp8):
    """Byte offsets past 32 bits and contexts of many steps, against the
    formula in float64."""
    Hkv, D, B = 8, 128, 16
    Hq, NB = G * Hkv, (1 << 18) + 7 if not fp8 else (1 << 19) + 7       # 2^32 bytes of cache is 2^17 (2^18) blocks
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    ctxs, news = [20011, 7], [n, min(n, 7)]
    gen = torch.Generator(device="cuda").manual_seed(18)
    dt = torch.uint8 if fp8 else torch.bfloat16
    kc, vc = (torch.empty(NB, Hkv, B, D, dtype=dt, device="cuda") for _ in range(2))
    used = sum(-(-c // B) for c in ctxs)
    tables = torch.full((2, -(-ctxs[0] // B)), -1, dtype=torch.int32)
    ids = torch.randperm(used, generator=torch.Generator().manual_seed(1)).to(torch.int32) + NB - used
    tables[0] = ids[:-1]
    tables[1, 0] = ids[-1]
    for c in (kc, vc):
        x = torch.randn(used, Hkv, B, D, generator=gen, device="cuda")
        c[NB - used:] = (x * 40).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x.to(dt)
    T = sum(news)
    q = torch.randn(T, Hq, D, generator=gen, device="cuda").to(torch.bfloat16)
    start = torch.tensor([0, news[0], T], dtype=torch.int32, device="cuda")
    out = torch.empty(T, Hq, D, dtype=torch.float32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.pa_decode_multi(out, q, kc, vc, tables.cuda(), start, torch.tensor(ctxs, dtype=torch.int32, device="cuda"), n, B,
                        1 / math.sqrt(D), Hq, Hkv, D, ctxs[0], workspace=api.decode_multi_workspace(n, Hq, Hkv, D),
                        status=st, k_scale=K_SCALE if fp8 else None, v_scale=V_SCALE if fp8 else None)
    assert st.item() == 0
    E, W = (2.0 ** -11, 2.0 ** -11) if fp8 else (0.0, 2.0 ** -16)
    for s, C in enumerate(ctxs):
        def rows(c, scale):
            x = c[tables[s, :-(-C // B)].long().cuda()]
            x = x.view(torch.float8_e4m3fn).double() * scale if fp8 else x.double()
            return x.permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :C]
        K, V = rows(kc, K_SCALE), rows(vc, V_SCALE)
        lo, m = int(start[s]), news[s]
        x = q[lo:lo + m].double().view(m, Hkv, G, D)
        z = torch.einsum("nhgd,hcd->hgnc", x, K) / math.sqrt(D)
        size = torch.einsum("nhgd,hcd->hgnc", x.abs(), K.abs()).amax(-1) / math.sqrt(D)   # [h, g, n]
        see = torch.ones(m, C, dtype=torch.bool, device="cuda").tril(C - m)
        a = torch.softmax(z.masked_fill(~see, -math.inf), -1)
        want = torch.einsum("hgnc,hcd->nhgd", a, V)
        weight = torch.einsum("hgnc,hcd->nhgd", a, V.abs())
        tol = (2 * (E + 128 * 2.0 ** -24) * size + W + 2.0 ** -18).permute(2, 0, 1)[..., None] * weight * 2
        got = out[lo:lo + m].double().view(m, Hkv, G, D)
        assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol).max().item()


@pytest.mark.parametrize("n,G,fp8", UNITS)
def test_whole_units_per_block_whether_the_bound_or_the_lengths_tell(n, G, fp8):
    """Short contexts take a block per unit: known from max_context_len, or
    only from the lengths; one context too long for that among them."""
    Hkv, D, B = 2, 128, 16
    ctxs, news = [60, 700, 33, 1, 64], [n, 2, n - 1, 1, 0]
    q, kc, vc, tables, start, ctx = p = _problem(21, G * Hkv, Hkv, D, B, ctxs, news, fp8=fp8, gap=1)
    near = _run(p, G * Hkv, Hkv, D, B, n, fp8=fp8)
    _check(p, near, G * Hkv, Hkv, D, B, fp8=fp8)
    wide = np.concatenate([tables, np.full((len(ctxs), 300), -1, dtype=np.int32)], 1)
    far = _run((q, kc, vc, wide, start, ctx), G * Hkv, Hkv, D, B, n, fp8=fp8, max_ctx=5000)
    assert torch.equal(near.view(torch.int32), far.view(torch.int32))
    p = _problem(22, G * Hkv, Hkv, D, B, [60, 1400, 33, 1, 64], news, fp8=fp8, gap=1)
    _check(p, _run(p, G * Hkv, Hkv, D, B, n, fp8=fp8), G * Hkv, Hkv, D, B, fp8=fp8)


def test_a_call_without_a_workspace_takes_one_of_its_own():
    Hq, Hkv, D, B = 8, 2, 128, 16
    p = q, kc, vc, tables, start, ctx = _problem(23, Hq, Hkv, D, B, [2000, 70], [4, 3])
    want = _run(p, Hq, Hkv, D, B, 4)
    a = [q.cuda(), from_bits(kc), from_bits(vc)] + [torch.from_numpy(x).cuda() for x in (tables, start, ctx)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, side.cuda_stream):
        out = torch.zeros(q.shape, dtype=torch.float32, device="cuda")
        torch.cuda.synchronize()
        api.pa_decode_multi(out, *a, 4, B, 1 / math.sqrt(D), Hq, Hkv, D, 2000, stream=stream)
        torch.empty(1 << 20, dtype=torch.uint8, device="cuda").fill_(0xFF)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int32), want.view(torch.int32))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("Hkv,G,D,B,ctxs,news", [
    (1, 4, 128, 16, [30001], [4]),                            # one head's keys over every SM: hundreds of pieces
    (1, 8, 128, 16, [20005], [9]),                            # the same in units of 64 rows
    (1, 16, 128, 32, [20001], [9]),                           # and of 128 (E4M3: three of 64)
    (2, 4, 128, 8, [1150, 193, 16], [4, 3, 1]),               # twelve warps, whole units
    (2, 2, 64, 16, [1500, 129, 700], [3, 1, 8]),              # twelve warps, shares
    (3, 2, 128, 32, [1153, 1152, 200], [2, 2, 2]),            # a step past what is not split
])
def test_few_units_of_long_contexts(Hkv, G, D, B, ctxs, news, fp8):
    if fp8 and D != 128:
        D = 128
    p = _problem(24, G * Hkv, Hkv, D, B, ctxs, news, fp8=fp8, gap=1)
    _check(p, _run(p, G * Hkv, Hkv, D, B, max(news), fp8=fp8), G * Hkv, Hkv, D, B, fp8=fp8)


@pytest.mark.parametrize("n,G,fp8", UNITS)
@pytest.mark.parametrize("C", [1000, 6000])                 # in one block, and in many
@pytest.mark.parametrize("above", [6.0, 9.0, 11.0, 20.0])
def test_one_large_weight_and_a_long_tail_of_small_ones(n, G, fp8, above, C):
    """A key whose score is `above` over thousands of others': their weights,
    2^-9 to 2^-29 of the largest, are what the output is made of."""
    Hkv, D, B = 1, 128, 16
    q, kc, vc, tables, start, ctx = _problem(25, G * Hkv, Hkv, D, B, [C], [n], fp8=fp8)
    q = (0.25 * torch.sign(q.float()[:1, :1].expand_as(q))).to(torch.bfloat16)
    rng = np.random.default_rng(26)
    k = 0.02 * rng.standard_normal(kc.shape)
    v = 1.0 + 0.1 * rng.standard_normal(vc.shape)
    k[tables[0, 3], :, 5] = above / (0.25 * math.sqrt(D)) * np.sign(q.float()[0, 0].numpy())
    v[tables[0, 3], :, 5] = 0.0
    put = (lambda x, s: Q.quantize(x, s)) if fp8 else (lambda x, s: to_bits(torch.from_numpy(x).to(torch.bfloat16)))
    p = (q, put(k, K_SCALE), put(v, V_SCALE), tables, start, ctx)
    _check(p, _run(p, G * Hkv, Hkv, D, B, n, fp8=fp8), G * Hkv, Hkv, D, B, fp8=fp8)


@pytest.mark.parametrize("n,G,fp8", UNITS)
def test_a_head_with_one_element_far_above_the_others(n, G, fp8):
    """An element of q some 16384 times the others, which meets keys that are zero
    there: the scores are the others' alone."""
    Hkv, D, B, C = 2, 128, 16, 700
    q, kc, vc, tables, start, ctx = _problem(27, G * Hkv, Hkv, D, B, [C], [n], fp8=fp8)
    q[:, :, 17] = 16384.0
    kc[..., 17] = 0
    p = (q, kc, vc, tables, start, ctx)
    _check(p, _run(p, G * Hkv, Hkv, D, B, n, fp8=fp8), G * Hkv, Hkv, D, B, fp8=fp8)


@pytest.mark.parametrize("fp8,D,G", [(False, 64, 8), (False, 128, 16), (True, 128, 8)])
def test_units_of_many_rows_over_more_sequences_than_threads(fp8, D, G):
    Hkv, B = 1, 8
    rng = np.random.default_rng(28)
    news = [int(x) for x in rng.integers(0, 2, 700)]
    news[3] = 4 if G == 8 else 8
    ctxs = [int(max(1, n + rng.integers(0, 150))) for n in news]
    p = _problem(28, G * Hkv, Hkv, D, B, ctxs, news, fp8=fp8)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _run(p, G * Hkv, Hkv, D, B, max(news), torch.bfloat16, fp8=fp8, status=st)
    assert st.item() == 0
    _check(p, out, G * Hkv, Hkv, D, B, fp8=fp8)


def test_calls_from_two_threads_at_once():
    """The library is entered by both: the binding lets go of the interpreter
    during a call."""
    import threading
    Hkv, D, B = 2, 128, 16
    work = []
    for n, G, fp8 in UNITS[:4]:
        p = _problem(29, G * Hkv, Hkv, D, B, [900, 40], [n, 2], fp8=fp8)
        q, kc, vc, tables, start, ctx = p
        put = (lambda c: torch.from_numpy(c).cuda()) if fp8 else from_bits
        work.append((n, G, fp8, [q.cuda(), put(kc), put(vc)] + [torch.from_numpy(x).cuda() for x in (tables, start, ctx)],
                     _run(p, G * Hkv, Hkv, D, B, n, fp8=fp8)))
    torch.cuda.synchronize()
    wrong = []

    def calls(order):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(25):
                for n, G, fp8, a, want in order:
                    out = torch.empty_like(want)
                    api.pa_decode_multi(out, *a, n, B, 1 / math.sqrt(D), G * Hkv, Hkv, D, 900,
                                        k_scale=K_SCALE if fp8 else None, v_scale=V_SCALE if fp8 else None)
                    stream.synchronize()
                    if not torch.equal(out.view(torch.int32), want.view(torch.int32)):
                        wrong.append((n, G, fp8))

    threads = [threading.Thread(target=calls, args=(o,)) for o in (work, work[::-1])]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("kind", ["causal", "tree"])
def test_many_rows_over_contexts_of_one_tile(fp8, kind):
    """Prompts and chunks of up to 128 positions in few sequences: 16 rows at a time."""
    Hq, Hkv, D, B, ctxs, news = 16, 4, 128, 16, [64, 128, 33, 7], [64, 20, 33, 1]
    p = _problem(30, Hq, Hkv, D, B, ctxs, news, fp8=fp8, gap=2)
    mask = [0] * 2 + _trees(news, np.random.default_rng(31)) + [0] * 2 if kind == "tree" else None
    _check(p, _run(p, Hq, Hkv, D, B, 64, torch.bfloat16, mask, fp8, max_ctx=128), Hq, Hkv, D, B, mask, fp8)


def test_a_workspace_of_its_own_is_ordered_with_what_the_memory_was_before():
    """Memory freed on the current stream with work on it still to run does not become the workspace of a call on
    another stream; the default stream by its handle, too."""
    Hq, Hkv, D, B = 8, 2, 128, 16
    p = q, kc, vc, tables, start, ctx = _problem(32, Hq, Hkv, D, B, [2000, 70], [4, 3])
    want = _run(p, Hq, Hkv, D, B, 4)
    a = [q.cuda(), from_bits(kc), from_bits(vc)] + [torch.from_numpy(x).cuda() for x in (tables, start, ctx)]
    size = api.pa_decode_multi_workspace_size(4, Hq, Hkv, D)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    out = torch.zeros(q.shape, dtype=torch.float32, device="cuda")
    for current, stream in ((torch.cuda.current_stream(), side), (torch.cuda.current_stream(), side.cuda_stream), (other, 0)):
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(current):
            before = torch.empty(size, dtype=torch.uint8, device="cuda")
            torch.cuda._sleep(4_000_000)                     # about 2 ms
            before.fill_(0x5A)
            torch.cuda._sleep(4_000_000)
            kept = before.clone()
            del before
            api.pa_decode_multi(out, *a, 4, B, 1 / math.sqrt(D), Hq, Hkv, D, 2000, stream=stream)
        torch.cuda.synchronize()
        assert (kept == 0x5A).all()
        assert torch.equal(out.view(torch.int32), want.view(torch.int32))


@pytest.mark.parametrize("n,G,fp8", [u for u in UNITS if not u[2]])
@pytest.mark.parametrize("C", [70, 3000])
def test_infinite_values_of_the_context_reach_their_column_alone(n, G, fp8, C):
    """Positions before the new ones, which every row sees: the column of their KV head's rows is not finite (an
    infinity may become NaN), and everything else is what finite values give."""
    Hkv, D, B = 2, 128, 16
    p = _problem(33, G * Hkv, Hkv, D, B, [C, 200], [n, 3])
    q, kc, vc, tables, start, ctx = p
    clean = vc.copy()
    for j, h, d, bits in ((0, 0, 5, 0x7F80), (C - n - 1, 0, 64, 0xFF80), (C // 2, 1, 127, 0x7F80)):
        at = tables[0, j // B], h, j % B, d
        vc[at], clean[at] = bits, 0
    out = _run(p, G * Hkv, Hkv, D, B, n)
    odd = torch.zeros_like(out, dtype=torch.bool)
    odd[:n, :G, 5] = odd[:n, :G, 64] = odd[:n, G:, 127] = True
    assert torch.equal(~torch.isfinite(out), odd)
    fine = _run((q, kc, clean, tables, start, ctx), G * Hkv, Hkv, D, B, n)
    _check((q, kc, clean, tables, start, ctx), torch.where(odd, fine, out), G * Hkv, Hkv, D, B)


@pytest.mark.parametrize("n,G,fp8", UNITS)
@pytest.mark.parametrize("Hkv,B,ctxs", [
    (1, 16, [30001]),                                        # one head's keys over every SM: hundreds of pieces
    (2, 32, [20011, 7, 193, 2048]),
    (2, 8, [1150, 1, 640, 129, 4097, 768]),                  # whole units, and shares that end anywhere
    (8, 16, [500 + 411 * i for i in range(9)]),              # an even split of ragged contexts
])
def test_every_position_of_long_contexts_counts_once(n, G, fp8, Hkv, B, ctxs):
    """q of zero, so that every weight is the same, and a position's value 1 in one column of 128 drawn for it: an
    output is the share of its column among the positions that the row sees.  Value sums are whole numbers times the
    weights' power of two, and exact.  So are the sums of weights where a weight is 2^0; E4M3 caches and more than 16
    rows take it as 2^12 from an approximation good to 2^-22, and the chain of a thread's additions is C / 4 at most,
    each good to 2^-24; factor and division take 2^-22.  A stretch of 16 positions lost or taken twice is several
    times that, which is tested on the formula's side."""
    D, news = 128, [min(n, c) for c in ctxs]
    q, kc, vc, tables, start, ctx = _problem(34, G * Hkv, Hkv, D, B, ctxs, news, fp8=fp8)
    q.zero_()
    rng = np.random.default_rng(35)
    column = [rng.integers(0, D, (c, Hkv)) for c in ctxs]
    for s, c in enumerate(ctxs):
        j = np.arange(c)
        at = tables[s, j // B], slice(None), j % B
        vc[at] = 0
        for h in range(Hkv):
            vc[tables[s, j // B], h, j % B, column[s][:, h]] = 0x38 if fp8 else 0x3F80
    got = out_to_f64(_run((q, kc, vc, tables, start, ctx), G * Hkv, Hkv, D, B, n, fp8=fp8))
    by = V_SCALE if fp8 else 1.0
    by = float(np.float32(by))
    for s, c in enumerate(ctxs):
        for h in range(Hkv):
            hits = np.zeros((c, D))
            hits[np.arange(c), column[s][:, h]] = 1.0
            total = hits.cumsum(0)
            off = 2.0 ** -21 + c / 4 * 2.0 ** -24
            for i in range(news[s]):
                see = c - news[s] + i + 1
                want = by * total[see - 1] / see
                rows = got[start[s] + i, h * G:(h + 1) * G]
                assert (np.abs(rows - want) <= off * want).all(), (s, h, i, np.abs(rows / want - 1).max())
            if c > 2000:
                part = np.add.reduceat(hits, np.arange(0, c, 16))
                length = np.minimum(16, c - np.arange(0, c, 16))[:, None]
                for sign in (-1, 1):
                    moved = np.abs((total[-1] + sign * part) / (c + sign * length) * c / total[-1] - 1).max(1)
                    assert moved[:-1].min() > 4 * off
