"""pa_attend and pa_attend_scaled against the float64 oracle, at the sizes,
masks and lengths where they can go wrong."""
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

MASKS = ["causal", "window", "documents", "spans", "blank"]


def _visible(kind, ctxs, news, rng, gap=0):
    """[T, 2] intervals, or None; rows of `gap` before and behind the sequences' own hold junk."""
    if kind == "causal":
        return None
    rows = [[7, 3]] * gap
    for c, n in zip(ctxs, news):
        for p in range(c - n, c):
            if kind == "window":
                rows.append([p - 20, p + 1])                       # (below 0 for early positions)
            elif kind == "documents":
                rows.append([p // 11 * 11, p + 1])
            elif kind == "spans":
                rows.append([0, max(p + 1, min(p // 9 * 9 + 9, c + 4))])   # (past the context for some)
            else:
                lo = int(rng.integers(0, c))                       # any interval, empty ones among them
                rows.append([lo, lo + int(rng.integers(-3, c))])
    return np.array(rows + [[1, 0]] * gap, dtype=np.int32)


class Problem:
    """Filled slots up to each context, NaN in every other; `gap` rows of q and out belong to no sequence."""

    def __init__(self, seed, Hq, Hkv, D, B, ctxs, news, mask="causal", scaled=False, gap=0, cap=0.0, alibi=False, scale=None):
        rng = np.random.default_rng(seed)
        nblk = [-(-c // B) for c in ctxs]
        NB, MB = sum(nblk) + 4, max(nblk + [1]) + 1
        ids = rng.permutation(NB).astype(np.int32)
        self.tables, at = np.full((len(ctxs), MB), -1, dtype=np.int32), 0
        for s, n in enumerate(nblk):
            self.tables[s, :n] = ids[at:at + n]
            at += n
        if scaled:
            draw = lambda: rng.choice(np.delete(np.arange(256), [0x7F, 0xFF]), (NB, Hkv, B, D)).astype(np.uint8)  # noqa: E731
            self.ks, self.vs = (rng.integers(112, 119, (NB, Hkv)).astype(np.uint8) for _ in range(2))
        else:
            draw = lambda: to_bits(I.bf16_normal((NB, Hkv, B, D), int(rng.integers(1 << 30))))  # noqa: E731
            self.ks = self.vs = None
        self.kc, self.vc = draw(), draw()
        self.filled = np.zeros((NB, B), dtype=bool)
        for s, c in enumerate(ctxs):
            for j in range(nblk[s]):
                self.filled[self.tables[s, j], :min(B, c - j * B)] = True
        for c in (self.kc, self.vc):
            blk, off = np.where(~self.filled)
            c[blk, :, off] = 0x7F if scaled else 0x7FC0
        self.start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32) + gap
        T = int(self.start[-1]) + gap
        self.q = I.bf16_normal((T, Hq, D), seed + 1)
        self.ctx = np.array(ctxs, dtype=np.int32)
        self.visible = _visible(mask, ctxs, news, rng, gap)
        self.cap, self.scale = cap, 1 / math.sqrt(D) if scale is None else scale
        self.slopes = (2.0 ** (-8.0 * np.arange(1, Hq + 1) / Hq)).astype(np.float32) if alibi else None
        self.Hq, self.Hkv, self.D, self.B, self.most = Hq, Hkv, D, B, max(news)

    def run(self, out_dtype=torch.float32, status=None, workspace=None, stream=None, out=None):
        dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
        put = dev if self.ks is not None else from_bits
        out = torch.full(self.q.shape, float("nan"), dtype=out_dtype, device="cuda") if out is None else out
        api.pa_attend(out, self.q.cuda(), put(self.kc), put(self.vc), dev(self.tables), dev(self.start), dev(self.ctx), self.most,
                      self.B, self.scale, self.Hq, self.Hkv, self.D, int(self.ctx.max()), visible=dev(self.visible),
                      softcap=self.cap, slopes=dev(self.slopes), k_scales=dev(self.ks), v_scales=dev(self.vs),
                      workspace=workspace, status=status, stream=stream)
        return out

    def check(self, out):
        """|out - ref| within what the roundings inside allow.  A score is off
        by the operand roundings and the products' 32 bits, (E + 128 2^-24)
        (|q| . |k|) |scale| (bf16: q exact; E4M3 codes: q to f16, 2^-11), by the
        cap's evaluation, 2^-20 of the score (a polynomial's 6e-7 and roundings)
        and 2^-21 of the cap (1 - 2 / (e + 1), whose quotient's 2^-22.5 of e and
        half steps come to 2^-23 of 1), and by a bias's roundings, 2^-20 of it
        (prompts count distances up in at most 16 additions, 2^-24 each);
        a weight by that and its own rounding W (bf16: two terms, 2^-16; else
        f16, 2^-11); all doubled, as the normaliser moves too; an output by
        that times sum a |v|, and half a step of its type.  Values that f16
        staging rounds (below 2^-14) and weights below f16's steps: 2^-24 of
        the largest |v|."""
        kd, vd = self.kc, self.vc
        if self.ks is not None:
            kd, vd = Q.dequantize_scaled(kd, self.ks), Q.dequantize_scaled(vd, self.vs)
        args = (self.tables, self.start, self.ctx, self.scale, self.B, self.visible, self.cap, self.slopes)
        f64 = (lambda c: c) if self.ks is not None else A.bf16_to_f64
        want = A.paged_shaped(to_bits(self.q), kd, vd, *args)
        weight = A.paged_shaped(to_bits(self.q), f64(kd), np.abs(f64(vd)), *args)
        E, W = (2.0 ** -11 if self.ks is not None else 0.0), 2.0 ** -11
        got, qa = out_to_f64(out), np.abs(A.bf16_to_f64(to_bits(self.q)))
        covered = np.zeros(self.q.shape[0], dtype=bool)
        G, ka, va = self.Hq // self.Hkv, np.abs(f64(kd)), np.abs(f64(vd))
        for s in range(len(self.ctx)):
            K, V = A.gather_kv(ka, va, self.tables[s], int(self.ctx[s]), self.B)
            for r in range(self.start[s], self.start[s + 1]):
                covered[r] = True
                for g in range(self.Hq):
                    size = np.nanmax(K[g // G] @ qa[r, g]) * abs(self.scale) if len(K[0]) else 0.0   # (NaN: where nobody looks)
                    bias = 0.0 if self.slopes is None else float(self.slopes[g]) * int(self.ctx[s])
                    off = (E + 128 * 2.0 ** -24) * size + 2.0 ** -20 * min(size, self.cap) + 2.0 ** -21 * self.cap + 2.0 ** -20 * bias + 2.0 ** -22 * size
                    tol = 2 * (off + W) * weight[r, g] * 2 + 2.0 ** -24 * (np.nanmax(V[g // G]) if len(V[0]) else 0.0)
                    if out.dtype == torch.bfloat16:
                        tol = tol + 2.0 ** -8 * np.abs(want[r, g])
                    assert (np.abs(got[r, g] - want[r, g]) <= tol).all(), (s, r, g, np.abs(got[r, g] - want[r, g]).max(), tol.max())
        assert np.isnan(got[~covered]).all()                       # rows of no sequence are left as they were
        return want


CASES = [
    # Hq, Hkv, D, B, contexts, new tokens
    (4, 2, 64, 16, [2, 16, 17, 38], [1, 2, 3, 1]),
    (32, 8, 128, 16, [1, 65, 300, 1000], [1, 4, 4, 2]),            # 16 rows
    (8, 8, 128, 8, [8, 9, 70, 513], [8, 1, 5, 7]),                 # G = 1, 8-position blocks
    (8, 4, 64, 32, [31, 64, 200], [16, 3, 9]),                     # 32 rows
    (32, 2, 128, 16, [40, 129], [3, 9]),                           # G = 16: 144 rows
    (16, 2, 64, 8, [61, 12], [20, 12]),                            # a whole prompt of 12
    (2, 1, 128, 32, [2500], [2]),                                  # one head: the keys over many blocks
    (4, 1, 128, 16, [150, 400, 33], [150, 131, 1]),                # prompts and chunks: tiles of 128 rows
    (2, 2, 64, 8, [333, 140], [333, 29]),
    (16, 2, 128, 8, [200, 77], [9, 30]),                           # 64 rows of 8-position blocks
    (8, 2, 128, 32, [300, 1500], [20, 41]),
]


@pytest.mark.parametrize("Hq,Hkv,D,B,ctxs,news", CASES)
@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("cap,alibi", [(0.0, False), (3.0, False), (0.0, True), (20.0, True)])
def test_attend_equals_the_oracle(Hq, Hkv, D, B, ctxs, news, mask, cap, alibi):
    p = Problem(Hq + D + B, Hq, Hkv, D, B, ctxs, news, mask, gap=2, cap=cap, alibi=alibi)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = p.run(torch.bfloat16 if alibi else torch.float32, status=st)
    assert st.item() == 0
    p.check(out)


@pytest.mark.parametrize("Hq,Hkv,D,B,ctxs,news", [c for c in CASES if c[2] == 128])
@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("cap,alibi", [(0.0, False), (5.0, True)])
def test_scaled_attend_equals_the_oracle(Hq, Hkv, D, B, ctxs, news, mask, cap, alibi):
    p = Problem(Hq + B, Hq, Hkv, D, B, ctxs, news, mask, scaled=True, gap=1, cap=cap, alibi=alibi)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = p.run(torch.bfloat16 if alibi else torch.float32, status=st)
    assert st.item() == 0
    p.check(out)


def _dense(p, take):
    """Rows `take` of p's outputs in float64 on the GPU, and sums of a |v| beside them, by the definition."""
    f64 = (lambda c, s: Q.dequantize_scaled(c, s)) if p.ks is not None else (lambda c, s: A.bf16_to_f64(c))
    K, V = (torch.from_numpy(f64(c, s)).cuda() for c, s in ((p.kc, p.ks), (p.vc, p.vs)))
    G, out, size = p.Hq // p.Hkv, [], []
    for r in take:
        s = int(np.searchsorted(p.start, r, side="right")) - 1
        C, pos = int(p.ctx[s]), int(p.ctx[s]) - int(p.start[s + 1]) + r
        lo, hi = (0, pos + 1) if p.visible is None else (max(0, int(p.visible[r][0])), min(C, int(p.visible[r][1])))
        ids = torch.from_numpy(p.tables[s][:-(-C // p.B)]).long().cuda()
        k, v = (x[ids].transpose(0, 1).reshape(p.Hkv, -1, p.D)[:, lo:max(hi, lo)] for x in (K, V))
        x = torch.einsum("hgd,hjd->hgj", p.q[r].double().cuda().view(p.Hkv, G, p.D), k) * p.scale
        if p.cap:
            x = p.cap * torch.tanh(x / p.cap)
        if p.slopes is not None:
            far = (torch.arange(lo, max(hi, lo), device="cuda") - pos).abs()
            x = x - torch.from_numpy(p.slopes).double().cuda().view(p.Hkv, G, 1) * far
        w = x.softmax(-1)
        out.append(torch.einsum("hgj,hjd->hgd", w, v).reshape(p.Hq, p.D))
        size.append(torch.einsum("hgj,hjd->hgd", w, v.abs()).reshape(p.Hq, p.D))
    return torch.stack(out), torch.stack(size)


PROMPTS = [
    # Hq, Hkv, D, B, sequences, the longest context, the most new tokens: enough of them for the prefill kernel's items
    (32, 8, 128, 16, 24, 300, 131),
    (16, 16, 64, 8, 12, 700, 700),
    (8, 8, 128, 32, 20, 900, 300),
    (64, 8, 128, 8, 16, 260, 100),
]


@pytest.mark.parametrize("Hq,Hkv,D,B,S,longest,most", PROMPTS)
@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("cap,alibi,scaled", [(0.0, False, False), (3.0, False, False), (20.0, True, False), (0.0, True, True),
                                              (30.0, False, True), (0.0, False, True)])
def test_prompts_equal_the_definition(Hq, Hkv, D, B, S, longest, most, mask, cap, alibi, scaled):
    """Tolerances as Problem.check's, with the largest |q| . |k| bounded by the products of the rows' sums and largest elements."""
    if scaled and D != 128:
        pytest.skip("E4M3 caches have heads of 128")
    rng = np.random.default_rng(S + most)
    ctxs = [int(c) for c in rng.integers(1, longest + 1, S)]
    ctxs[0], ctxs[1] = longest, 1
    news = [min(c, int(n)) for c, n in zip(ctxs, rng.integers(1, most + 1, S))]
    news[0] = most
    p = Problem(Hq + S, Hq, Hkv, D, B, ctxs, news, mask, scaled=scaled, gap=1, cap=cap, alibi=alibi)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = p.run(status=st)
    assert st.item() == 0
    assert torch.isnan(out[0]).all() and torch.isnan(out[-1]).all()
    take = sorted({1, 2, int(p.start[1]) - 1, int(p.start[1]), int(p.start[-1]) - 1} | set(rng.integers(1, int(p.start[-1]), 60).tolist()))
    want, weight = _dense(p, take)
    kd, vd = (Q.dequantize_scaled(c, s) if scaled else A.bf16_to_f64(c) for c, s in ((p.kc, p.ks), (p.vc, p.vs)))
    qa = p.q[take].double().cuda().abs()
    size = (qa.sum(-1) * float(np.nanmax(np.abs(kd))) * p.scale)[..., None]
    bias = 0.0 if p.slopes is None else torch.from_numpy(p.slopes).double().cuda()[:, None] * longest
    off = ((2.0 ** -11 if scaled else 0.0) + 128 * 2.0 ** -24) * size + 2.0 ** -20 * size.clamp(max=cap) + 2.0 ** -21 * cap + \
        2.0 ** -20 * bias + 2.0 ** -22 * size
    tol = 2 * (off + 2.0 ** -11) * weight * 2 + 2.0 ** -24 * float(np.nanmax(np.abs(vd)))
    got = out[take].double()
    assert ((got - want).abs() <= tol).all(), (got - want).abs().max()
    # and far within it on the whole: weights' roundings are as often up as down
    assert (got - want).norm() <= 2.0 ** -9 * weight.norm()


@pytest.mark.parametrize("scaled", [False, True], ids=["bf16", "scaled"])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_values_that_are_not_finite_in_prompts(scaled, out_dtype):
    S, n = 24, 131
    p = Problem(1, 32, 8, 128, 16, [300] * S, [n] * S, "window", scaled=scaled)
    p.visible[:, 0], p.visible[:, 1] = 100, 200
    clean = p.run(out_dtype)
    bad = 0x7F if scaled else 0xFF80                               # NaN, or an infinity
    for j in list(range(0, 100, 9)) + [99, 200, 201, 255, 299]:
        for c in (p.kc, p.vc):
            c[p.tables[:, j // 16], :, j % 16] = bad
    assert torch.equal(p.run(out_dtype), clean)
    p = Problem(1, 32, 8, 128, 16, [300] * S, [n] * S, "window", scaled=scaled)
    p.visible[:, 0], p.visible[:, 1] = 100, 200
    p.visible[::2, 1] = 250
    before = p.run(out_dtype)
    p.vc[p.tables[3, 220 // 16], 1, 220 % 16, 5] = bad             # seen by the even tokens of one sequence, in one KV head
    after = p.run(out_dtype)
    got, want = ~torch.isfinite(after), torch.zeros(after.shape, dtype=torch.bool, device="cuda")
    rows = torch.arange(3 * n, 4 * n, device="cuda")
    want[rows[rows % 2 == 0], 4:8, 5] = True
    assert torch.equal(got, want) and torch.equal(after[~got], before[~got])
    if not scaled:                                                 # and values past fp16's range beside it
        p.vc[p.tables[3, 150 // 16], 1, 150 % 16, 7] = 0x4880      # 2^18
        wide = p.run(out_dtype)
        assert torch.equal(~torch.isfinite(wide), want)
        off = (wide[3 * n:4 * n, 4:8, 8:].float() - before[3 * n:4 * n, 4:8, 8:].float()).abs().max()
        assert off <= 2 * 2.0 ** -10 * 5 + 2.0 ** -7 * before.abs().max() * (out_dtype == torch.bfloat16)   # (weights in two terms instead of f16)


@pytest.mark.parametrize("scaled", [False, True], ids=["bf16", "scaled"])
@pytest.mark.parametrize("scale", [0.0, -0.07, 1.5])
@pytest.mark.parametrize("news", [[1, 4], [70, 40]], ids=["few", "many"])
def test_other_scales(scaled, scale, news):
    p = Problem(9, 8, 2, 128, 16, [100, 333], news, "window", scaled=scaled, cap=30.0, scale=scale)
    p.check(p.run())


@pytest.mark.parametrize("scaled", [False, True], ids=["bf16", "scaled"])
@pytest.mark.parametrize("news", [[1], [4], [70]], ids=["1", "4", "70"])
def test_a_shifted_start_of_the_positions_seen(scaled, news):
    """Windows that begin at every offset within tiles and blocks, ends likewise."""
    for lo in range(0, 40, 7):
        for length in (1, 2, 15, 16, 17, 130):
            p = Problem(lo + length, 4, 1, 128, 8, [300], news, "window", scaled=scaled)
            p.visible[:] = [lo, lo + length]
            p.check(p.run())


@pytest.mark.parametrize("scaled", [False, True], ids=["bf16", "scaled"])
@pytest.mark.parametrize("news", [[3, 2], [80, 17]], ids=["few", "many"])
def test_rows_that_see_nothing_are_zeros(scaled, news):
    p = Problem(4, 8, 2, 128, 16, [90, 200], news, "window", scaled=scaled, alibi=True)
    p.visible[1] = [50, 50]
    p.visible[2] = [60, 2]
    p.visible[news[0]:] = [500, 600]                               # past the second sequence's context: all of its rows
    out = p.run()
    p.check(out)
    assert (out[1:3] == 0).all() and (out[news[0]:] == 0).all()


@pytest.mark.parametrize("scaled", [False, True], ids=["bf16", "scaled"])
@pytest.mark.parametrize("news", [[3], [8], [90], [150]], ids=["3", "8", "90", "150"])
@pytest.mark.parametrize("empty", [(400, 400), (0, 0), (9, 3), (2000, 3000)])
def test_rows_that_see_nothing_beside_rows_that_see_all(scaled, news, empty):
    """Tiles that need no mask for the others."""
    p = Problem(4, 4, 1, 128, 16, [900], news, "window", scaled=scaled)
    p.visible[:, 0], p.visible[:, 1] = 0, 900
    p.visible[1] = empty
    p.visible[-1] = empty
    if empty == (2000, 3000):                                      # and NaN where nobody looks
        p.visible[::3, 0] = 20
        for c in (p.kc, p.vc):
            c[p.tables[0, 0], :, 3] = 0x7F if scaled else 0x7FC0
        p.visible[:, 0] = np.maximum(p.visible[:, 0], 4)
    out = p.run()
    p.check(out)
    assert (out[1] == 0).all() and (out[-1] == 0).all()


@pytest.mark.parametrize("scaled", [False, True], ids=["bf16", "scaled"])
@pytest.mark.parametrize("news", [[2], [7], [90]], ids=["2", "7", "90"])
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_what_a_token_does_not_see_does_not_reach_it(scaled, news, what):
    """NaN and infinities at positions outside a token's interval, in keys and values, within the context."""
    if scaled and what == "inf":
        pytest.skip("E4M3 has no infinity")
    p = Problem(11, 8, 2, 128, 16, [300], news, "window", scaled=scaled)
    p.visible[:, 0], p.visible[:, 1] = 100, 200
    clean = p.run()
    bad = 0x7F if scaled else (0x7FC0 if what == "nan" else 0xFF80)
    for j in list(range(0, 100, 9)) + [99, 200, 201, 255, 299]:
        for c in (p.kc, p.vc):
            c[p.tables[0, j // 16], :, j % 16] = bad
    assert torch.equal(p.run(), clean)
    # a value within the interval of the even tokens only: they alone get it
    p = Problem(11, 8, 2, 128, 16, [300], news, "window", scaled=scaled)
    p.visible[:, 0], p.visible[:, 1] = 100, 200
    p.visible[::2, 1] = 250
    before = p.run()
    p.vc[p.tables[0, 220 // 16], 1, 220 % 16, 5] = bad
    after = p.run()
    got = ~torch.isfinite(after)
    want = torch.zeros_like(got)
    want[::2, 4:, 5] = True
    assert torch.equal(got, want)
    assert torch.equal(after[~got], before[~got])


@pytest.mark.parametrize("news", [[1, 1, 1], [9, 40, 64]], ids=["one", "many"])
def test_equal_scales_are_the_cache_of_one_scale(news):
    """A block-scaled cache whose scales are all 2^-5: within both roundings of pa_decode_multi_fp8."""
    p = Problem(5, 8, 2, 128, 16, [64, 257, 900], news, scaled=True)
    p.ks[:], p.vs[:] = 122, 122
    out = p.run()
    ref = torch.empty_like(out)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    api.pa_decode_multi(ref, p.q.cuda(), dev(p.kc), dev(p.vc), dev(p.tables), dev(p.start), dev(p.ctx), p.most, 16, p.scale, 8, 2,
                        128, 900, k_scale=2.0 ** -5, v_scale=2.0 ** -5)
    p.check(out)
    p.check(ref)


def test_scales_of_very_different_blocks():
    """Values whose blocks' scales are 2^24 apart, and blocks of zeros with the least scale."""
    p = Problem(6, 4, 1, 128, 8, [120], [1], scaled=True)
    p.ks[:] = 115
    for j in range(15):
        p.vs[p.tables[0, j]] = 130 if j == 7 else 106
    p.vc[p.tables[0, 7], :, :, 1:] = 0                             # the largest scale, values in one column
    p.vc[p.tables[0, 3]] = 0
    p.vs[p.tables[0, 3]] = 0
    p.kc[p.tables[0, 4]] = 0
    p.ks[p.tables[0, 4]] = 0
    out = p.run()
    p.check(out)


@pytest.mark.parametrize("scaled", [False, True], ids=["bf16", "scaled"])
@pytest.mark.parametrize("most", [1, 6, 100])
def test_calls_are_repeatable_captured_and_on_other_streams(scaled, most):
    p = Problem(7, 8, 2, 128, 16, [700, 1300, 100], [most, min(most, 5), most], "window", scaled=scaled, cap=8.0)
    first = p.run()
    p.check(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = p.run()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again, first)
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    put = dev if scaled else from_bits
    args = [p.q.cuda(), put(p.kc), put(p.vc), dev(p.tables), dev(p.start), dev(p.ctx), p.most, 16, p.scale, 8, 2, 128, 1300]
    kw = dict(visible=dev(p.visible), softcap=8.0, k_scales=dev(p.ks), v_scales=dev(p.vs))
    out = torch.full_like(first, float("nan"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.pa_attend(out, *args, **kw)                            # (a workspace of the graph's own)
    out.fill_(float("nan"))
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)


@pytest.mark.parametrize("scaled", [False, True], ids=["bf16", "scaled"])
@pytest.mark.parametrize("news", [[2, 3, 1], [70, 3, 40]], ids=["few", "many"])
def test_bad_inputs_are_flagged(scaled, news):
    p = Problem(8, 4, 1, 128, 16, [90, 60, 200], news, scaled=scaled)
    want = p.run()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    p.ctx[1] = 2                                                   # less than its new tokens: not computed
    out = p.run(status=st)
    assert st.item() == api.PA_DEV_BAD_CONTEXT
    a, b = p.start[1], p.start[2]
    assert torch.equal(out[:a], want[:a]) and torch.equal(out[b:], want[b:]) and torch.isnan(out[a:b]).all()
    p.ctx[1], st[0] = 60, 0
    most, p.most = p.most, max(n for n in news if n < p.most)      # more new tokens than the call allows: not computed
    out = p.run(status=st)
    p.most = most
    left = torch.isnan(out).all(-1).all(-1)
    assert st.item() == api.PA_DEV_BAD_CONTEXT
    assert left.tolist() == [n == most for n in news for _ in range(n)]
    # (another kernel may take the smaller call: each within 2 (2^-11 + 2^-11) of sums of a |v|, by the roundings of weights and q)
    top = float(np.nanmax(np.abs(Q.dequantize_scaled(p.vc, p.vs) if scaled else A.bf16_to_f64(p.vc))))
    assert (out[~left] - want[~left]).abs().max() <= 2 * 4 * 2.0 ** -11 * top
    p.tables[0, 1] = 1 << 20                                       # outside the pool: flagged, the others as they were
    st.zero_()
    out = p.run(status=st)
    assert st.item() == api.PA_DEV_BAD_BLOCK_ID
    assert torch.equal(out[a:], want[a:])


def test_long_contexts_and_offsets_past_31_bits():
    """Contexts of 70,000 positions whose blocks lie past 2^31 elements of the cache; a window within them."""
    B, D = 32, 128
    NB = (1 << 31) // (B * D) + 2200
    kc = torch.zeros(NB, 1, B, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    n = -(-70000 // B)
    tables = torch.arange(NB - n, NB, dtype=torch.int32, device="cuda")[None].contiguous()
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn(n * B, D, generator=g, device="cuda").bfloat16()
    v = torch.randn(n * B, D, generator=g, device="cuda").bfloat16()
    kc[NB - n:] = k.view(n, 1, B, D)
    vc[NB - n:] = v.view(n, 1, B, D)
    for new in (1, 40):
        q = torch.randn(new, 4, D, generator=g, device="cuda").bfloat16()
        i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        for lo in (0, 61234):
            vis = torch.stack([i32(*[lo] * new), i32(*range(70000 - new + 1, 70001))], 1).contiguous()
            out = torch.empty(new, 4, D, dtype=torch.float32, device="cuda")
            api.pa_attend(out, q, kc, vc, tables, i32(0, new), i32(70000), new, B, 0.088, 4, 1, D, 70000, visible=vis, softcap=20.0)
            s = 20 * torch.tanh(q.double() @ k.double().T * 0.088 / 20)
            j = torch.arange(n * B, device="cuda")
            s = s.masked_fill((j < vis[:, :1, None]) | (j >= vis[:, 1:, None]), -math.inf)
            want = s.softmax(-1) @ v.double()
            # weights to f16 at the most: 2 2^-11, doubled, of sums of a |v|; the scores' 32 bits
            tol = 2 ** -9 * (s.softmax(-1) @ v.double().abs()) + 2e-5
            assert ((out - want).abs() <= tol).all()


def test_a_step_planned_written_and_attended():
    """A run of the operators, as a serving step makes it: planned on the GPU, projections turned by three axes and appended
    to a block-scaled cache, attended within a window."""
    Hq, Hkv, D, B, S, MB = 8, 2, 128, 16, 3, 16
    NB = S * MB + 3
    dev = "cuda"
    rows, row_lens, row_blocks = (torch.tensor(x, dtype=torch.int32, device=dev) for x in ([2, 0, 1], [0] * S, [0] * S))
    row_tables = torch.full((S, MB), -1, dtype=torch.int32, device=dev)
    free, count = torch.randperm(NB, device=dev).int(), torch.tensor([NB], dtype=torch.int32, device=dev)
    bt, ctx = torch.empty_like(row_tables), torch.empty(S, dtype=torch.int32, device=dev)
    start = torch.empty(S + 1, dtype=torch.int32, device=dev)
    kc = torch.full((NB, Hkv, B, D), 0x7F, dtype=torch.uint8, device=dev)
    vc = torch.full_like(kc, 0x7F)
    ks = torch.full((NB, Hkv), 255, dtype=torch.uint8, device=dev)   # nothing reads a scale that no append has written
    vs = torch.full_like(ks, 255)
    table, gain = api.rope_table(500, D), torch.ones(D, device=dev)
    axes = api.rope_axes([24, 20, 20])
    g = torch.Generator(device=dev).manual_seed(3)
    for new in ([100, 7, 33], [1, 1, 1], [4, 1, 2]):
        T = sum(new)
        pos, slots = torch.empty(T, dtype=torch.int32, device=dev), torch.empty(T, dtype=torch.int64, device=dev)
        api.pa_plan_step(bt, ctx, start, pos, slots, rows, torch.tensor(new, dtype=torch.int32, device=dev), row_lens, row_tables,
                         row_blocks, free, count, B, NB)
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device=dev).mul_(3).bfloat16()
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
        q_out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        api.pa_qk_norm_rope_cache_scaled(q_out, kc, vc, ks, vs, q, k, v, torch.stack([pos, pos // 2, pos // 3]), slots, table,
                                         axes=axes, q_weight=gain, k_weight=gain, status=st)
        vis = torch.stack([(pos - 49).clamp(min=0), pos + 1], 1)
        out = torch.empty(T, Hq, D, dtype=torch.float32, device=dev)
        api.pa_attend(out, q_out, kc, vc, bt, start, ctx, max(new), B, D ** -0.5, Hq, Hkv, D, MB * B, visible=vis, softcap=30.0,
                      k_scales=ks, v_scales=vs, status=st)
        assert st.item() == 0
        row_lens[rows.long()] += torch.tensor(new, dtype=torch.int32, device=dev)
        h = lambda t: t.cpu().numpy()  # noqa: E731
        kd, vd = Q.dequantize_scaled(h(kc), h(ks)), Q.dequantize_scaled(h(vc), h(vs))
        want = A.paged_shaped(to_bits(q_out.cpu()), kd, vd, h(bt), h(start), h(ctx), D ** -0.5, B, h(vis), 30.0)
        # norm-1 rows times sqrt(D): |q| |k| scale <= sqrt(D); q to f16, weights to f16, both sides of the quotient
        assert np.abs(out_to_f64(out) - want).max() <= 4 * (2.0 ** -11 * (D ** 0.5 + 1)) * np.nanmax(np.abs(vd))


@pytest.mark.parametrize("scaled", [False, True], ids=["bf16", "scaled"])
@pytest.mark.parametrize("most", [1, 20, 300])
def test_two_calls_at_once(scaled, most):
    """Two graphs of their own workspaces, replayed side by side on two streams."""
    problems = [Problem(11 + i, 8, 2, 128, 16, [900 + i, 400], [most, max(1, most // 3)], "window", scaled=scaled, cap=5.0 * i)
                for i in range(2)]
    want = [p.run() for p in problems]
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    graphs, outs, held = [], [], []
    for p, w in zip(problems, want):
        p.check(w)
        put = dev if scaled else from_bits
        args = [p.q.cuda(), put(p.kc), put(p.vc), dev(p.tables), dev(p.start), dev(p.ctx), p.most, 16, p.scale, 8, 2, 128, 901]
        kw = dict(visible=dev(p.visible), softcap=p.cap, k_scales=dev(p.ks), v_scales=dev(p.vs),
                  workspace=api.attend_workspace(2, p.most, p.tables.shape[1], 16, 8, 2, 128, scaled))
        out = torch.full_like(w, float("nan"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.pa_attend(out, *args, **kw)
        graphs.append(g)
        outs.append(out)
        held.append((args, kw))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        assert torch.equal(out, w)


def test_tensors_of_wrong_type_shape_place_or_layout_are_refused():
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    b = lambda *s: z(*s, dt=torch.bfloat16)  # noqa: E731
    u = lambda *s: z(*s, dt=torch.uint8)  # noqa: E731
    f = lambda *s: z(*s, dt=torch.float32)  # noqa: E731
    attend = dict(out=b(3, 4, 64), q=b(3, 4, 64), k_cache=b(2, 2, 16, 64), v_cache=b(2, 2, 16, 64), block_tables=z(1, 2),
                  query_start=z(2), context_lens=z(1), max_query_len=3, block_size=16, scale=0.125, n_q_heads=4,
                  n_kv_heads=2, d_head=64, max_context_len=32)
    scaled = dict(attend, out=b(3, 4, 128), q=b(3, 4, 128), k_cache=u(2, 2, 16, 128), v_cache=u(2, 2, 16, 128), d_head=128,
                  k_scales=u(2, 2), v_scales=u(2, 2))
    mrope = dict(q_out=b(3, 4, 64), k_cache=b(2, 2, 16, 64), v_cache=b(2, 2, 16, 64), q=b(3, 4, 64), k=b(3, 2, 64),
                 v=b(3, 2, 64), positions=z(2, 3), axes=[0, 1] * 16, slot_mapping=z(3).long() - 1, cos_sin=f(9, 64))
    codes = dict(k_cache=u(2, 2, 16, 64), v_cache=u(2, 2, 16, 64), k_scales=u(2, 2), v_scales=u(2, 2))
    rope = dict(mrope, **codes)
    append = dict(codes, k=b(3, 2, 64), v=b(3, 2, 64), slot_mapping=z(3).long() - 1)
    for fn, good, cases in (
            (api.pa_attend, attend, [
                (dict(out=z(3, 4, 64)), TypeError, "out must be bfloat16"), (dict(q=b(3, 2, 64)), ValueError, "q must be"),
                (dict(q=b(3, 64, 4).transpose(1, 2)), ValueError, "q must be contiguous"),
                (dict(visible=z(3)), ValueError, "visible must be"), (dict(visible=z(3, 2).long()), TypeError, "visible must be"),
                (dict(visible=z(2, 3).t()), ValueError, "visible must be contiguous"),
                (dict(slopes=f(2)), ValueError, "slopes must be"), (dict(slopes=b(4)), TypeError, "slopes must be"),
                (dict(slopes=f(4).cpu()), ValueError, "slopes must be a CUDA tensor"), (dict(softcap="x"), TypeError, None),
                (dict(k_scales=u(2, 2)), ValueError, "go together"),
                (dict(k_scales=u(2, 2), v_scales=u(2, 2)), TypeError, "k_cache must be torch.uint8"),
                (dict(workspace=z(16)), TypeError, "workspace must be torch.uint8"),
                (dict(workspace=u(16)), api.PAError, None)]),
            (api.pa_attend, scaled, [
                (dict(k_cache=b(2, 2, 16, 128)), TypeError, "k_cache must be torch.uint8"),
                (dict(k_scales=u(2)), ValueError, "k_scales must be"), (dict(v_scales=f(2, 2)), TypeError, "v_scales must be"),
                (dict(v_scales=u(2, 4)[:, ::2]), ValueError, "v_scales must be contiguous")]),
            (api.pa_qk_norm_mrope_cache, mrope, [
                (dict(positions=z(3)), ValueError, "positions must"), (dict(positions=z(2, 4)), ValueError, "positions must be"),
                (dict(axes=[0] * 31), ValueError, "axes must have"), (dict(axes=[0, 300] * 16), ValueError, None),
                (dict(axes="x" * 32), TypeError, None), (dict(axes=[2, 1] * 16), api.PAError, None),
                (dict(axes=None), TypeError, "axes must be"), (dict(k_scale=0.1), ValueError, "go together")]),
            (api.pa_qk_norm_rope_cache_scaled, rope, [
                (dict(k_cache=b(2, 2, 16, 64)), TypeError, "k_cache must be torch.uint8"),
                (dict(axes=None), ValueError, "positions must"), (dict(v_scales=u(1, 2)), ValueError, "v_scales must be"),
                (dict(v_scales=None), TypeError, "v_scales must be")]),
            (api.pa_reshape_and_cache_scaled, append, [
                (dict(k=b(3, 4, 64)), ValueError, "k must be"), (dict(v=b(4, 2, 64)), ValueError, "v must be"),
                (dict(slot_mapping=z(3)), TypeError, "slot_mapping must be"), (dict(k_scales=None), TypeError, "k_scales must be"),
                (dict(v_cache=u(2, 2, 64, 16).transpose(2, 3)), ValueError, "v_cache must be contiguous")])):
        assert fn(**good) == api.PA_OK
        for change, error, text in cases:
            with pytest.raises(error, match=text):
                fn(**dict(good, **change))
    torch.cuda.synchronize()


@pytest.mark.parametrize("scaled,lengths", [(False, range(1000, 1100)), (True, range(1100, 1200)), (False, [1500] * 99 + [3])])
def test_one_unit_for_most_blocks(scaled, lengths):
    """400 units of nearly one length, too long for a rule by length; and one that is much shorter."""
    p = Problem(21, 4, 4, 128, 16, list(lengths), [1] * 100, scaled=scaled, cap=20.0)
    p.check(p.run())


@pytest.mark.parametrize("scaled", [False, True], ids=["bf16", "scaled"])
@pytest.mark.parametrize("news", [[4, 1], [6, 30], [70, 12], [300, 40]])
def test_intervals_at_the_ends_of_32_bits(scaled, news):
    p = Problem(31, 8, 2, 128, 16, [n + 230 for n in news], news, "window", scaled=scaled)
    lo, hi = -2 ** 31, 2 ** 31 - 1
    ends = [(lo, None), (0, hi), (lo, lo), (hi, lo), (hi, hi), (lo, hi), (100, hi), (lo, 7), (lo + 1, 0)]
    for t in range(len(p.visible)):
        a, b = ends[t % len(ends)]
        p.visible[t] = a, p.visible[t, 1] if b is None else b
    p.check(p.run())


@pytest.mark.parametrize("cap", [1e-40, 1e-20, 1e-7, 1e-3, 1e5, 1e30, 3e38])
@pytest.mark.parametrize("news", [[3], [30], [300]])
def test_caps_of_any_size(cap, news):
    """Among them rows of q, and keys, that are zeros: scores of 0."""
    p = Problem(32, 8, 2, 128, 16, [n + 230 for n in news], news, cap=cap)
    q = to_bits(p.q).copy()
    q[::2] = 0
    p.q = from_bits(q).cpu()
    p.check(p.run())


@pytest.mark.parametrize("cap", [1e-40, 1e-7, 1.0])
@pytest.mark.parametrize("news", [[3], [30], [300]])
def test_scores_of_zero_under_a_cap(cap, news):
    p = Problem(33, 8, 2, 128, 16, [n + 230 for n in news], news, cap=cap)
    p.q = torch.zeros_like(p.q)
    p.check(p.run())


def test_the_readmes_prompt_with_an_image():
    """Within the roundings of check(), a score's size bounded by the largest norms."""
    import os
    import re
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    with open(path) as f:
        (code,) = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    x = {}
    exec(compile(code, "README.md", "exec"), x)
    torch.cuda.synchronize()
    n, nb = x["n"], -(-x["n"] // x["B"])
    k, v = (Q.dequantize_scaled(x[c][:nb].cpu().numpy(), x[s][:nb].cpu().numpy()) for c, s in (("codes", "scales"), ("v_codes", "v_scales")))
    q = to_bits(x["q_turned"])
    args = (x["table"].cpu().numpy(), [0, n], [n], x["scale"], x["B"], x["visible"].cpu().numpy(), 50.0)
    want, weight = A.paged_shaped(q, k, v, *args), A.paged_shaped(q, k, np.abs(v), *args)
    size = x["scale"] * np.linalg.norm(A.bf16_to_f64(q), axis=-1).max() * np.linalg.norm(k, axis=-1).max()
    off = (2.0 ** -11 + 128 * 2.0 ** -24 + 2.0 ** -20) * size + 2.0 ** -21 * 50 + 2.0 ** -11
    assert (np.abs(out_to_f64(x["seen"]) - want) <= 4 * off * weight + 2.0 ** -8 * np.abs(want)).all()
