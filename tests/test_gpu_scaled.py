"""pa_qk_norm_mrope_cache, pa_qk_norm_rope_cache_scaled and
pa_reshape_and_cache_scaled against the oracle."""
import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import quant as Q
from oracle import step as S
from _gpu_util import to_bits

pytestmark = pytest.mark.gpu

api = pytest.importorskip("paged_kv_cache_124_gb300.api")
from paged_kv_cache_124_gb300 import inputs as I  # noqa: E402

dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731


def _qkv(T, Hq, Hkv, D, seed, packed=True):
    if not packed:
        return [I.bf16_normal((T, h, D), seed + i).cuda() for i, h in enumerate((Hq, Hkv, Hkv))]
    qkv = I.bf16_normal((T, (Hq + 2 * Hkv) * D), seed).cuda()
    return [x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 1)]


def _expected(x, gain, eps, pos, axes, interleaved):
    """Exact rows and their tolerance before the final rounding, [T, H, D]:
    32-bit sums and products put a turned element within 2^-19 (|a| + |b|) of
    its pair (a, b): at most 19 additions and 8 products and factors in a row
    and the table's own rounding, each 2^-24, and rsqrt's two units."""
    x64 = A.bf16_to_f64(to_bits(x))
    y, tol = np.empty_like(x64), np.empty_like(x64)
    rot = 2 * len(axes)
    for t in range(x64.shape[0]):
        at = [int(pos[a, t]) for a in axes]
        for h in range(x64.shape[1]):
            y[t, h] = S.norm_rope(x64[t, h], gain, eps, at, rot, interleaved)
            pair = np.abs(S.norm_rope(x64[t, h], gain, eps, 0, rot, interleaved))
            c = np.arange(rot // 2)
            i, j = (2 * c, 2 * c + 1) if interleaved else (c, c + rot // 2)
            pair[i] = pair[j] = pair[i] + pair[j]
            tol[t, h] = pair * 2.0 ** -19
    return y, tol


def _close(got, want, tol, half_step, smallest=0.0):
    off = np.abs(got - want)
    assert (off <= tol + half_step * (np.abs(want) + tol) + smallest).all(), off.max()


def _gains(rng, D, norm):
    return [(1 + 0.2 * rng.standard_normal(D)).astype(np.float32) if norm else None for _ in range(2)]


AXES = [
    # T, Hq, Hkv, D, B, sections, in turn, interleaved pairs, norm
    (1, 32, 8, 128, 16, [16, 24, 24], False, False, True),
    (37, 4, 2, 64, 8, [8, 12, 12], False, True, True),
    (19, 8, 1, 128, 32, [24, 20, 20], True, False, True),
    (23, 2, 2, 64, 16, [3, 5], False, False, False),               # 16 of 64 elements turn, two axes
    (11, 16, 4, 128, 16, [64], False, False, True),                # one axis
    (9, 6, 3, 64, 16, [1, 2, 3, 18], True, True, False),           # four
    (900, 16, 8, 128, 16, [16, 24, 24], True, False, True),        # tokens enough for a thread's angles to serve all heads
]


@pytest.mark.parametrize("T,Hq,Hkv,D,B,sections,turn,inter,norm", AXES)
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_several_axes_equal_the_oracle(T, Hq, Hkv, D, B, sections, turn, inter, norm, fp8):
    rng = np.random.default_rng(T + D)
    few = min(T, 40)                                               # rows that the oracle's loops look at
    if T > 40:
        T *= 7
    q, k, v = _qkv(T, Hq, Hkv, D, T)
    NB = -(-T // B) + 3
    slots = rng.permutation(NB * B)[:T].astype(np.int64)
    axes = api.rope_axes(sections, turn)
    pos = rng.integers(0, 3000, (len(sections), T)).astype(np.int32)
    qw, kw = _gains(rng, D, norm)
    kc = torch.full((NB, Hkv, B, D), 0x5A, dtype=torch.uint8, device="cuda") if fp8 else \
        torch.full((NB, Hkv, B, D), 7.5, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    out = torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.pa_qk_norm_mrope_cache(out, kc, vc, q, k, v, dev(pos), axes, dev(slots), api.rope_table(3000, 2 * sum(sections)),
                               q_weight=dev(qw), k_weight=dev(kw), eps=1e-5, interleaved=inter, status=st,
                               **(dict(k_scale=0.013, v_scale=0.021) if fp8 else {}))
    assert st.item() == 0
    at = np.sort(rng.permutation(T)[:few])
    want, tol = _expected(q[at], qw, 1e-5, pos[:, at], axes, inter)
    _close(A.bf16_to_f64(to_bits(out[at])), want, tol, 2.0 ** -8)
    want, tol = _expected(k[at], kw, 1e-5, pos[:, at], axes, inter)
    rows = lambda c: c.cpu().permute(0, 2, 1, 3).reshape(NB * B, Hkv, D)[torch.from_numpy(slots)]  # noqa: E731
    if fp8:
        s = float(np.float32(0.013))
        want, tol = np.clip(want / s, -448, 448), tol / s + np.abs(want / s) * 2.0 ** -23
        _close(Q.e4m3_to_f64(rows(kc).numpy()[at]), want, tol, 2.0 ** -4, 2.0 ** -10)
        assert np.array_equal(rows(vc).numpy(), Q.quantize(v.float().cpu().numpy(), np.float32(0.021)))
    else:
        _close(A.bf16_to_f64(to_bits(rows(kc)[at])), want, tol, 2.0 ** -8)
        assert np.array_equal(to_bits(rows(vc)), to_bits(v))


@pytest.mark.parametrize("sections", [[64], [16, 24, 24]])
def test_equal_positions_on_all_axes_are_one_axis(sections):
    T, Hq, Hkv, D, B = 300, 8, 2, 128, 16
    q, k, v = _qkv(T, Hq, Hkv, D, 3)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 7
    slots, table, w = torch.arange(T, device="cuda"), api.rope_table(2200, D), torch.ones(D, device="cuda")
    caches = [torch.zeros(20, Hkv, B, D, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    one, many = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    api.pa_qk_norm_rope_cache(one, caches[0], caches[1], q, k, v, pos, slots, table, q_weight=w, k_weight=w)
    api.pa_qk_norm_mrope_cache(many, caches[2], caches[3], q, k, v, pos.repeat(len(sections), 1), api.rope_axes(sections), slots,
                               table, q_weight=w, k_weight=w)
    assert torch.equal(one, many) and torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


def test_a_token_with_a_bad_position_on_any_axis():
    T, Hq, Hkv, D, B = 6, 4, 2, 128, 16
    q, k, v = _qkv(T, Hq, Hkv, D, 3)
    pos = np.array([[1, 2, 3, 4, 5, 6], [1, -1, 3, 50, 5, 6], [1, 2, 3, 4, 49, -7]], dtype=np.int32)
    kc = torch.zeros(2, Hkv, B, D, dtype=torch.bfloat16, device="cuda")
    vc, out = kc.clone(), torch.full((T, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.pa_qk_norm_mrope_cache(out, kc, vc, q, k, v, dev(pos), api.rope_axes([16, 24, 24]), torch.arange(T, device="cuda"),
                               api.rope_table(50, D), status=st)
    assert st.item() == api.PA_DEV_BAD_POSITION
    assert [bool((out[t] == 3.0).all()) for t in range(T)] == [False, True, False, True, False, True]
    assert [bool((vc[0, :, t] != 0).any()) for t in range(T)] == [True, False, True, False, True, False]


# ---------------------------------------------------------------------------
# block-scaled caches
# ---------------------------------------------------------------------------

def _slots(runs, B, NB, rng):
    """Slots of runs of (first offset, tokens), each in blocks of its own from a shuffled pool."""
    ids, at, slots = rng.permutation(NB), 0, []
    for off, n in runs:
        j = off + np.arange(n)
        slots.append(ids[at + j // B] * B + j % B)
        at += (off + n - 1) // B + 1
    assert at <= NB
    return np.concatenate(slots).astype(np.int64)


RUNS = [
    [(0, 1)], [(5, 1)], [(0, 3), (7, 1), (2, 2)],
    [(0, 100)], [(3, 77), (0, 32), (7, 1), (1, 33)],
    [(i % 8, 1) for i in range(40)],                               # a decode batch
]


@pytest.mark.parametrize("runs", RUNS, ids=["one", "one more", "few", "prompt", "mixed", "decodes"])
@pytest.mark.parametrize("Hkv,D,B", [(2, 128, 16), (1, 64, 8), (3, 64, 32), (8, 128, 32), (2, 128, 8), (4, 64, 16)])
def test_append_of_values_as_they_are(runs, Hkv, D, B):
    """Bit for bit: no arithmetic comes before the codes.  Over blocks with codes and scales of every size."""
    rng = np.random.default_rng(Hkv + D + B)
    T, NB = sum(n for _, n in runs), sum((o + n - 1) // B + 1 for o, n in runs) + 2
    slots = _slots(runs, B, NB, rng)
    k, v = (I.bf16_normal((T, Hkv, D), 5 + i) for i in range(2))
    k = (k.float() * torch.from_numpy(2.0 ** rng.integers(-12, 12, (T, Hkv, 1))).float()).bfloat16()
    codes = [rng.integers(0, 256, (NB, Hkv, B, D)).astype(np.uint8) for _ in range(2)]
    scales = [rng.integers(100, 130, (NB, Hkv)).astype(np.uint8) for _ in range(2)]
    got = [dev(c) for c in codes + scales]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    strided = torch.cat([k.cuda(), v.cuda()], 1)                   # views of one projection's rows
    api.pa_reshape_and_cache_scaled(*got, strided[:, :Hkv], strided[:, Hkv:], dev(slots), status=st)
    assert st.item() == 0
    for c, s, x, gc, gs in zip(codes, scales, (k, v), got[:2], got[2:]):
        Q.append_scaled(c, s, A.bf16_to_f64(to_bits(x)), slots.tolist(), B)
        assert np.array_equal(gs.cpu().numpy(), s)
        g = gc.cpu().numpy()
        nan = (c & 0x7F) == 0x7F
        assert np.array_equal(nan, (g & 0x7F) == 0x7F) and np.array_equal(g[~nan], c[~nan])


def test_append_special_values():
    """Zeros, infinities, NaN, the values about a power of two's limits, and the smallest."""
    Hkv, D, B = 1, 64, 8
    rows = [[0.0], [1e-38], [448.0], [449.0], [447.0, float("inf")], [float("nan"), 3.0], [float("-inf")], [3.0e38], [-1e-41, 0.0]]
    x = torch.zeros(len(rows), Hkv, D)
    for t, r in enumerate(rows):
        x[t, 0, :len(r)] = torch.tensor(r)
    x = x.bfloat16()
    slots = np.arange(len(rows), dtype=np.int64) * B               # a block each
    codes, scales = np.full((len(rows), Hkv, B, D), 0x11, np.uint8), np.full((len(rows), Hkv), 200, np.uint8)
    got = [dev(codes), dev(codes), dev(scales), dev(scales)]
    api.pa_reshape_and_cache_scaled(*got, x.cuda(), x.cuda(), dev(slots))
    Q.append_scaled(codes, scales, A.bf16_to_f64(to_bits(x)), slots.tolist(), B)
    for i in range(2):
        g = got[i].cpu().numpy()
        nan = (codes & 0x7F) == 0x7F
        assert np.array_equal(got[2 + i].cpu().numpy(), scales)
        assert np.array_equal(nan, (g & 0x7F) == 0x7F) and np.array_equal(g[~nan], codes[~nan])


@pytest.mark.parametrize("span", [1, 3, 40])
def test_appending_as_tokens_come_keeps_within_a_step_of_their_values(span):
    """A block filled in calls of `span` tokens of growing size: each element within E4M3's half step of its value, and what
    growing scales cut: half of E4M3's smallest step, of the scale at each growth, which are powers of two."""
    Hkv, D, B, T = 2, 128, 16, 64
    x = (I.bf16_normal((T, Hkv, D), 3).float() * 2.0 ** (torch.arange(T)[:, None, None] % 16 / 2)).bfloat16()
    kc, vc = (torch.zeros(5, Hkv, B, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((5, Hkv), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    for t in range(0, T, span):
        part = x[t:t + span].cuda()
        api.pa_reshape_and_cache_scaled(kc, vc, ks, vs, part, -part, torch.arange(t, min(t + span, T), device="cuda") + B)
    got = Q.dequantize_scaled(kc.cpu().numpy(), ks.cpu().numpy())[1:].transpose(0, 2, 1, 3).reshape(T, Hkv, D)
    want = x.double().numpy()
    step = 2.0 ** (ks.cpu().numpy()[1:].astype(float) - 127 - 9)      # of the smallest codes
    assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + np.repeat(step, B, 0)[:, :, None]).all()
    assert torch.equal(vc[1:] ^ 0x80, kc[1:]) and torch.equal(vs, ks)   # (nothing was written to block 0)


@pytest.mark.parametrize("T,Hq,Hkv,D,B,sections,inter,norm,packed,runs", [
    (1, 32, 8, 128, 16, None, False, True, True, [(3, 1)]),
    (37, 4, 2, 64, 8, None, False, True, True, [(0, 20), (5, 9), (2, 8)]),
    (40, 8, 1, 128, 32, [16, 24, 24], False, True, True, [(0, 35), (31, 1), (9, 4)]),
    (23, 2, 2, 64, 16, [8, 8], True, True, False, [(1, 1), (0, 1), (7, 21)]),
    (30, 16, 4, 128, 16, [24, 20, 20], False, False, True, [(15, 30)]),
])
def test_norm_rope_append_equals_the_oracle(T, Hq, Hkv, D, B, sections, inter, norm, packed, runs):
    rng = np.random.default_rng(T + Hq)
    q, k, v = _qkv(T, Hq, Hkv, D, 2 * T, packed)
    axes = [0] * (D // 2) if sections is None else list(api.rope_axes(sections, T == 30))
    pos = rng.integers(0, 900, (max(axes) + 1, T)).astype(np.int32)
    NB = sum((o + n - 1) // B + 1 for o, n in runs) + 2
    slots = _slots(runs, B, NB, rng)
    qw, kw = _gains(rng, D, norm)
    codes = [rng.integers(0, 0x7F, (NB, Hkv, B, D)).astype(np.uint8) for _ in range(2)]
    scales = [rng.integers(112, 120, (NB, Hkv)).astype(np.uint8) for _ in range(2)]
    kc, vc, ks, vs = (dev(c) for c in codes + scales)
    out = torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.pa_qk_norm_rope_cache_scaled(out, kc, vc, ks, vs, q, k, v, dev(pos[0] if sections is None else pos), dev(slots),
                                     api.rope_table(900, 2 * len(axes)), axes=None if sections is None else axes, q_weight=dev(qw),
                                     k_weight=dev(kw), eps=1e-5, interleaved=inter, status=st)
    assert st.item() == 0
    want, tol = _expected(q, qw, 1e-5, pos, axes, inter)
    _close(A.bf16_to_f64(to_bits(out)), want, tol, 2.0 ** -8)
    Q.append_scaled(codes[1], scales[1], A.bf16_to_f64(to_bits(v)), slots.tolist(), B)
    assert np.array_equal(vs.cpu().numpy(), scales[1]) and np.array_equal(vc.cpu().numpy(), codes[1])
    want, tol = _expected(k, kw, 1e-5, pos, axes, inter)
    Q.append_scaled(codes[0], scales[0], want, slots.tolist(), B)
    assert np.array_equal(ks.cpu().numpy(), scales[0])             # (no largest value lies within its tolerance of a limit)
    rows = lambda c: c.transpose(0, 2, 1, 3).reshape(NB * B, Hkv, D)  # noqa: E731
    unit = np.repeat(2.0 ** (scales[0].astype(float) - 127), B, 0)[slots][:, :, None]
    _close(rows(Q.e4m3_to_f64(kc.cpu().numpy()))[slots], want / unit, tol / unit, 2.0 ** -4, 2.0 ** -10)
    keep = np.setdiff1d(np.arange(NB * B), slots)
    assert np.array_equal(rows(kc.cpu().numpy())[keep], rows(codes[0])[keep])   # the blocks' other codes, coded again or as they were


@pytest.mark.parametrize("T,Hkv,D,B", [(5003, 9, 128, 16), (5003, 4, 64, 32), (2003, 9, 128, 32), (900, 5, 64, 8)])
def test_many_tokens_are_the_same_in_calls_of_few(T, Hkv, D, B):
    """Calls of sizes that divide the work in other ways, over heads that fill no whole share, against calls of a few hundred tokens."""
    Hq = 2 * Hkv
    q, k, v = _qkv(T, Hq, Hkv, D, 1)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    NB = T // B + 9
    slots = torch.randperm(NB, device="cuda")[torch.arange(T, device="cuda") // B] * B + torch.arange(T, device="cuda") % B
    table, w = api.rope_table(T, D), torch.rand(D, device="cuda") + 0.5

    def run(parts):
        g = torch.Generator(device="cuda").manual_seed(1)
        c = [torch.randint(0, 127, (NB, Hkv, B, D), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
        s = [torch.full((NB, Hkv), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
        out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        for x in parts:
            api.pa_qk_norm_rope_cache_scaled(out[x], *c, *s, q[x], k[x], v[x], pos[x], slots[x], table, q_weight=w, k_weight=w)
        return [out] + c + s

    whole = run([slice(0, T)])
    for a, b in zip(whole, run([slice(t, min(t + 320, T)) for t in range(0, T, 320)])):   # (whole blocks)
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,Hkv,D,B", [(5003, 8, 128, 16), (3003, 15, 128, 32), (6003, 7, 64, 8), (16003, 2, 128, 16)])
def test_many_tokens_of_heads_that_fill_their_tiles_or_do_not(T, Hkv, D, B):
    test_many_tokens_are_the_same_in_calls_of_few(T, Hkv, D, B)


def test_padding_bad_positions_and_bad_slots_of_the_append():
    T, Hq, Hkv, D, B, NB = 9, 4, 2, 128, 16, 4
    q, k, v = _qkv(T, Hq, Hkv, D, 3)
    pos = np.array([4, -1, 49, 50, 7, 8, -5, 9, 10], dtype=np.int32)
    slots = np.array([0, 1, 16, 17, -1, NB * B, 5, 32, 33], dtype=np.int64)
    kc, vc = (torch.zeros(NB, Hkv, B, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((NB, Hkv), 9, dtype=torch.uint8, device="cuda") for _ in range(2))
    out = torch.full((T, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.pa_qk_norm_rope_cache_scaled(out, kc, vc, ks, vs, q, k, v, dev(pos), dev(slots), api.rope_table(50, D), status=st)
    assert st.item() == api.PA_DEV_BAD_POSITION | api.PA_DEV_BAD_SLOT
    assert [bool((out[t] == 3.0).all()) for t in range(T)] == [False, True, False, True, False, False, True, False, False]
    written = (vc != 0).any(-1).any(1).cpu()
    assert torch.nonzero(written).tolist() == [[0, 0], [1, 0], [2, 0], [2, 1]]
    assert (vs[3] == 9).all() and (vs[:3] != 9).all()


def test_captured_appends_replay():
    T, Hq, Hkv, D, B = 4, 8, 2, 128, 16
    q, k, v = _qkv(T, Hq, Hkv, D, 8)
    pos, slots = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int64, device="cuda")
    kc, vc = (torch.zeros(T, Hkv, B, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((T, Hkv), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    out, table = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda"), api.rope_table(64, D)
    call = lambda o, c: api.pa_qk_norm_rope_cache_scaled(o, *c, q, k, v, pos, slots, table)  # noqa: E731
    slots.fill_(-1)
    call(out, (kc, vc, ks, vs))                                    # (loads the kernel; writes nothing)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out, (kc, vc, ks, vs))
    eager, plain = [t.clone() for t in (kc, vc, ks, vs)], torch.empty_like(out)
    for step in range(20):
        q.normal_(), k.normal_().mul_(1 + step % 7), v.normal_()
        pos.fill_(step)
        slots.copy_(torch.arange(T, device="cuda") * B + step % B)
        g.replay()
        call(plain, eager)
        assert torch.equal(out, plain) and all(torch.equal(a, b) for a, b in zip((kc, vc, ks, vs), eager))
