"""pa_attend and pa_attend_scaled where something outside of what a row sees
could reach it: scales, table entries and values of blocks that are not its
own, and magnitudes at the ends of what the kernels' types hold."""
import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import quant as Q
from _gpu_util import from_bits, out_to_f64, to_bits
from test_gpu_attend import Problem

pytestmark = pytest.mark.gpu

api = pytest.importorskip("paged_kv_cache_124_gb300.api")


def _rows(p):
    """(row, sequence, position, first seen, end of the seen) of p's new tokens."""
    for s, C in enumerate(p.ctx.tolist()):
        for r in range(p.start[s], p.start[s + 1]):
            pos = C - int(p.start[s + 1]) + r
            lo, hi = (0, pos + 1) if p.visible is None else (max(0, int(p.visible[r][0])), min(C, int(p.visible[r][1])))
            yield r, s, pos, lo, max(hi, lo)


def _want(p, r, s, pos, lo, hi):
    """Row r by the definition in float64, [Hq, D]; sums of a |v| beside it; the largest sum of |q| |k| and |v| that it sees."""
    G, at = p.Hq // p.Hkv, np.arange(lo, hi)
    blk, off = p.tables[s][at // p.B], at % p.B
    f64 = lambda c, s: A.bf16_to_f64(c[blk, :, off]) if s is None else \
        Q.e4m3_to_f64(c[blk, :, off]) * 2.0 ** (s[blk].astype(float) - 127)[..., None]  # noqa: E731
    k, v = f64(p.kc, p.ks), f64(p.vc, p.vs)                         # [hi - lo, Hkv, D]
    q = A.bf16_to_f64(to_bits(p.q[r:r + 1]))[0].reshape(p.Hkv, G, p.D)
    x = np.einsum("hgd,jhd->hgj", q, k) * p.scale
    size = np.einsum("hgd,jhd->hgj", np.abs(q), np.abs(k)).max(-1) * abs(p.scale)
    if p.cap:
        x = p.cap * np.tanh(x / p.cap)
    if p.slopes is not None:
        x = x - p.slopes.astype(float).reshape(p.Hkv, G, 1) * np.abs(pos - at)
    w = np.exp(x - x.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    out, weight = (np.einsum("hgj,jhd->hgd", w, y).reshape(p.Hq, p.D) for y in (v, np.abs(v)))
    return out, weight, size.reshape(p.Hq, 1), np.abs(v).max((0, 2)).repeat(G)[:, None]


def _check(p, out, least=2.0 ** -24, smallest=0.0, take=lambda rows: rows):
    """Problem.check's tolerances, with magnitudes of what a row sees alone:
    weights below f16's steps, `least` of the largest |v|; what is below
    `smallest` may be lost.  Returns the norms of all errors and all sums of
    a |v|."""
    got, off, all_ = out_to_f64(out), 0.0, 0.0
    E = 2.0 ** -11 if p.ks is not None else 0.0                    # codes' q to f16
    for r, s, pos, lo, hi in take(list(_rows(p))):
        if lo == hi:
            assert (got[r] == 0).all()
            continue
        want, weight, size, top = _want(p, r, s, pos, lo, hi)
        bias = 0.0 if p.slopes is None else np.abs(p.slopes[:, None].astype(float)) * (hi - lo)
        s_off = (E + 128 * 2.0 ** -24 + 2.0 ** -22) * size + 2.0 ** -20 * np.minimum(size, p.cap) + 2.0 ** -21 * p.cap + 2.0 ** -20 * bias
        tol = 2 * (s_off + 2.0 ** -11) * weight * 2 + least * top + smallest
        if out.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * np.abs(want)
        bad = np.abs(got[r] - want)
        assert (bad <= tol).all(), (r, s, bad.max(), (bad / tol).max())
        off, all_ = off + (bad ** 2).sum(), all_ + (weight ** 2).sum()
    return off ** 0.5, all_ ** 0.5


def _few(n):
    rng = np.random.default_rng(0)
    return lambda rows: [rows[i] for i in sorted(rng.choice(len(rows), min(n, len(rows)), replace=False))]


def _to_other_place(p, block, to):
    """Swap two blocks of the pool."""
    for c in (p.kc, p.vc, p.ks, p.vs):
        if c is not None:
            c[[block, to]] = c[[to, block]]
    a, b = p.tables == block, p.tables == to
    p.tables[a], p.tables[b] = to, block


def _unused(p):
    return np.setdiff1d(np.arange(len(p.kc)), p.tables[p.tables >= 0])


@pytest.mark.parametrize("Hq,new", [(4, 1), (4, 2), (16, 1), (4, 8)])
@pytest.mark.parametrize("mask,cap", [("causal", 0.0), ("window", 0.0), ("causal", 5.0)])
@pytest.mark.parametrize("byte", [255, 200])
@pytest.mark.parametrize("B", [8, 16, 32])
def test_scales_of_blocks_that_are_not_its_own(Hq, new, mask, cap, byte, B):
    """Contexts that end in either half of a tile of 16 positions; block 0 and all others of no sequence hold no scale, or a large one."""
    for ctx in (1, 5, 8, 9, 17, 24, 45, 52):
        p = Problem(3, Hq, 1, 128, B, [ctx], [min(new, ctx)], mask, scaled=True, cap=cap)
        _to_other_place(p, 0, _unused(p)[0])
        p.ks[_unused(p)] = p.vs[_unused(p)] = byte
        _check(p, p.run())


@pytest.mark.parametrize("B", [8, 16, 32])
def test_a_sequence_as_its_tokens_come(B):
    """Appended and attended token by token, then four by four, in a pool whose unwritten scales are none."""
    Hq, Hkv, D, n = 8, 2, 128, 70
    g = torch.Generator(device="cuda").manual_seed(B)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda").mul_(2).bfloat16()  # noqa: E731
    NB = n // B + 3
    kc, vc = (torch.full((NB, Hkv, B, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((NB, Hkv), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    table = (NB - 1 - torch.arange(NB - 1, device="cuda")).int()[None].contiguous()   # (block 0 is of no sequence)
    done = 0
    for new in [1] * 34 + [4] * 9:
        at = torch.arange(done, done + new, device="cuda")
        api.pa_reshape_and_cache_scaled(kc, vc, ks, vs, draw(new, Hkv, D), draw(new, Hkv, D), table[0].long()[at // B] * B + at % B)
        done += new
        p = Problem(1, Hq, Hkv, D, B, [done], [new], scaled=True)
        p.kc, p.vc, p.ks, p.vs, p.tables, p.q = (*(t.cpu().numpy() for t in (kc, vc, ks, vs, table)), draw(new, Hq, D).cpu())
        _check(p, p.run())


@pytest.mark.parametrize("scaled", [False, True], ids=["bf16", "scaled"])
@pytest.mark.parametrize("mask", ["causal", "window"])
def test_sequences_without_new_tokens_cost_and_flag_nothing(scaled, mask):
    """Beside prompts: one without new tokens whose table is not there, and one that is flagged for more of them than positions."""
    news = [131, 0, 131, 40] + [131] * 20
    p = Problem(6, 32, 8, 128, 16, [300] * 24, news, mask, scaled=scaled)
    clean = p.run()
    p.tables[1] = -1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert torch.equal(p.run(status=st), clean) and st.item() == 0
    p.ctx[3], p.tables[3] = 39, -1
    out = p.run(status=st)
    rest = torch.ones(len(out), dtype=torch.bool, device="cuda")
    rest[p.start[3]:p.start[4]] = False
    assert st.item() == api.PA_DEV_BAD_CONTEXT and torch.equal(out[rest], clean[rest]) and torch.isnan(out[~rest]).all()


def _unseen_blocks(p, low, high):
    """Of the first sequence: blocks that hold none of the positions low .. high - 1."""
    n = -(-int(p.ctx[0]) // p.B)
    return [j for j in range(n) if (j + 1) * p.B <= low or j * p.B >= high]


@pytest.mark.parametrize("scaled", [False, True], ids=["bf16", "scaled"])
@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("S,new", [(1, 2), (1, 7), (1, 60), (24, 131)])
def test_blocks_that_no_token_sees_need_not_be_there(scaled, B, S, new):
    """A cache that frees blocks behind its window, and ones in front of what is seen: entries of -1 or past the pool, codes
    and scales of whoever has the block now.  Nothing is flagged, and not a bit changes."""
    for low, high in ((100, 200), (139, 141), (8, 299), (127, 129), (256, 300), (0, 3)):
        p = Problem(5, 8, 2, 128, B, [300] * S, [new] * S, "window", scaled=scaled)
        p.visible[:] = [low, high]
        p.visible[::3, 0] = min(low + 1, high - 1)
        clean = p.run()
        _check(p, clean, take=_few(12))
        gone = _unseen_blocks(p, low, high)
        for s in range(S):
            ids = p.tables[s][gone]
            p.kc[ids] = p.vc[ids] = 0x7F if scaled else 0x7FC0
            if scaled:
                p.ks[ids] = p.vs[ids] = 255
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        assert torch.equal(p.run(status=st), clean) and st.item() == 0
        for s in range(S):
            p.tables[s][gone] = [-1 if j % 2 else len(p.kc) + j for j in gone]
        assert torch.equal(p.run(status=st), clean) and st.item() == 0


@pytest.mark.parametrize("scaled", [False, True], ids=["bf16", "scaled"])
@pytest.mark.parametrize("S,new", [(2, 2), (2, 60), (24, 131)])
def test_a_table_that_no_token_looks_at(scaled, S, new):
    p = Problem(5, 8, 2, 128, 16, [300] * S, [new] * S, "window", scaled=scaled)
    p.visible[p.start[1]:p.start[2]] = [200, 200]
    clean, st = p.run(), torch.zeros(1, dtype=torch.int32, device="cuda")
    p.tables[1] = -1
    assert torch.equal(p.run(status=st), clean) and st.item() == 0 and (clean[p.start[1]:p.start[2]] == 0).all()


@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("S,new", [(1, 2), (1, 4), (1, 40), (24, 131)])
@pytest.mark.parametrize("apart", [20, 40, 90])
def test_documents_whose_scales_are_far_apart(B, S, new, apart):
    """Two documents in a sequence, the values of one 2^apart of the other's: each as exact as by itself, whichever comes first."""
    for first in (False, True):
        p = Problem(7, 4, 1, 128, B, [300] * S, [new] * S, "window", scaled=True)
        cut = 160
        for s in range(S):
            p.vs[p.tables[s][:cut // B]] = 115 if first else 115 - apart
            p.vs[p.tables[s][cut // B:-(-300 // B)]] = 115 - apart if first else 115
        p.visible[::2], p.visible[1::2] = [0, cut], [cut, 300]
        p.visible[::4, 0], p.visible[::4, 1] = 150, 160            # (a few positions beside the other document's)
        _check(p, p.run(), take=_few(12))
    for s in range(S):                                             # beside the largest scale that there is
        p.vs[p.tables[s][:cut // B]], p.vs[p.tables[s][cut // B:-(-300 // B)]] = 115, 254
    _check(p, p.run(), take=lambda rows: _few(12)([r for r in rows if r[4] <= cut]))


@pytest.mark.parametrize("S,new", [(1, 2), (1, 4), (1, 40), (24, 131)])
@pytest.mark.parametrize("byte", [1, 2, 6, 7, 20])
def test_values_of_the_smallest_scales(S, new, byte):
    """Elements below fp32's smallest normal number, 2^-126, may be taken for zeros."""
    p = Problem(8, 4, 1, 128, 8, [300] * S, [new] * S, "window", scaled=True)
    p.vs[:] = byte
    _check(p, p.run(), smallest=2.0 ** -126, take=_few(12))
    p.vs[p.tables[0][:20]] = 0                                     # beside blocks of the least
    p.visible[:] = [100, 300]
    _check(p, p.run(), smallest=2.0 ** -126 + 448 * 2.0 ** -127, take=_few(12))


@pytest.mark.parametrize("Hq,Hkv,D,B,S,new", [(32, 8, 128, 16, 24, 131), (16, 16, 64, 8, 24, 260), (4, 2, 128, 16, 2, 3), (16, 2, 128, 32, 2, 20)])
@pytest.mark.parametrize("shift", [8, 18, 30])
@pytest.mark.parametrize("rows", ["all", "some", "mixed"])
def test_small_values(Hq, Hkv, D, B, S, new, shift, rows):
    """Values 2^-shift of a normal deviate's, at all positions, at every fifth, or the second half of each head: relative to the
    largest of the positions that are seen, as any others (below 2^-14 f16 has steps of 2^-24, half of which is 2^-15 of
    2^-10, from where on a position's are taken for f16)."""
    p = Problem(9, Hq, Hkv, D, B, [300] * S, [new] * S, "spans")
    v = from_bits(p.vc, "cpu").float()
    if rows == "all":
        v *= 2.0 ** -shift
    elif rows == "some":
        v[:, :, ::5] *= 2.0 ** -shift
    else:
        v[..., D // 2:] *= 2.0 ** -shift
    p.vc = to_bits(v.bfloat16())
    if rows == "some":                                             # rows that see one such position alone
        p.visible[::2, 0] = p.visible[::2, 1] - 1
    _check(p, p.run(), least=2.0 ** -15, take=_few(16))


@pytest.mark.parametrize("scaled", [False, True], ids=["bf16", "scaled"])
@pytest.mark.parametrize("S,new", [(1, 2), (1, 7), (1, 90), (24, 131)])
@pytest.mark.parametrize("cap,alibi", [(3.0, False), (20.0, True), (50.0, False)])
def test_unseen_keys_do_not_change_how_a_cap_is_taken(scaled, S, new, cap, alibi):
    """Keys that no token sees, made large, not finite or zeros: not a bit of the rows changes."""
    p = Problem(10, 8, 2, 128, 16, [300] * S, [new] * S, "window", scaled=scaled, cap=cap, alibi=alibi)
    p.visible[:] = [103, 197]
    clean = p.run()
    _check(p, clean, take=_few(12))
    hidden = [j for j in range(300) if not 103 <= j < 197]
    for bits in ([0x7E, 0xFE], [0x7F, 0x7F], [0, 0]) if scaled else ([0x4780, 0xC780], [0x7F80, 0x7FC0], [0, 0]):   # 2^16; inf, NaN
        for s in range(S):
            for n, j in enumerate(hidden):
                p.kc[p.tables[s][j // 16], :, j % 16] = bits[n % 2]
        assert torch.equal(p.run(), clean)


@pytest.mark.parametrize("scaled", [False, True], ids=["bf16", "scaled"])
@pytest.mark.parametrize("S,new", [(1, 40), (24, 131)])
@pytest.mark.parametrize("alibi", [False, True])
def test_keys_that_others_see_do_not_change_how_a_cap_is_taken(scaled, S, new, alibi):
    """The even tokens see keys that the odd ones do not: large, they are far beyond the cap; the odd ones' rows keep every bit."""
    p = Problem(13, 8, 2, 128, 16, [300] * S, [new] * S, "window", scaled=scaled, cap=30.0, alibi=alibi)
    p.visible[:] = [0, 150]
    p.visible[::2] = [0, 300]
    clean = p.run()
    for s in range(S):
        for j in range(150, 300, 7):
            p.kc[p.tables[s][j // 16], :, j % 16] = 0x7E if scaled else 0x4380      # 448, 2^8
    out = p.run()
    assert torch.equal(out[1::2], clean[1::2])
    _check(p, out, take=_few(12))


@pytest.mark.parametrize("scaled", [False, True], ids=["bf16", "scaled"])
@pytest.mark.parametrize("S,new,ctx", [(1, 2, 1 << 20), (1, 4, 1 << 20), (1, 40, 1 << 20), (64, 128, 1 << 18)])
@pytest.mark.parametrize("slope", [0.5, 0.0625])
def test_a_bias_over_positions_far_from_the_token(scaled, S, new, ctx, slope):
    """A token that sees a short interval far behind it, or ahead of it: the distance to all of the interval is no weight's
    concern, and takes no bits of the rest."""
    B, n = 16, 8
    p = Problem(11, 4, 1, 128, B, [n * B] * S, [1] * S, scaled=scaled)
    p.tables = np.ascontiguousarray(np.tile(p.tables[:, :n], (1, ctx // (n * B))))   # the same blocks again and again
    p.ctx[:] = ctx
    p.start = (np.arange(S + 1) * new).astype(np.int32)
    p.q = torch.randn(S * new, 4, 128, generator=torch.Generator().manual_seed(1)).bfloat16()
    p.most, p.slopes = new, np.full(4, slope, dtype=np.float32)
    p.visible = np.tile(np.array([[5, 60]], dtype=np.int32), (S * new, 1))
    p.visible[1::2] = [37, 131]
    out = p.run()
    off, weight = _check(p, out, take=_few(16))
    assert off <= 2.0 ** -10 * weight                              # weights' roundings, 2^-11 at the most, as often up as down
    p.visible[:] = [ctx - 60, ctx]                                 # ahead of some, about others
    off, weight = _check(p, p.run(), take=_few(16))
    assert off <= 2.0 ** -10 * weight


@pytest.mark.parametrize("scaled", [False, True], ids=["bf16", "scaled"])
@pytest.mark.parametrize("S,new", [(1, 4), (1, 90), (24, 131)])
@pytest.mark.parametrize("slope", [3e37, 1e30, -0.01])
def test_slopes_of_any_size(scaled, S, new, slope):
    """The nearest position alone where a slope is large; the farther the more where it is negative."""
    p = Problem(12, 4, 1, 128, 16, [300] * S, [new] * S, "window", scaled=scaled)
    p.slopes = np.full(4, slope, dtype=np.float32)
    p.visible[:] = [20, 100]
    out = p.run()
    if slope < 0:
        _check(p, out, take=_few(12))
    else:
        for r, s, pos, lo, hi in _few(12)(list(_rows(p))):
            want = _want(p, r, s, pos, hi - 1, hi)[0]
            assert (np.abs(out_to_f64(out[r]) - want) <= 2.0 ** -10 * np.abs(want)).all()


def test_a_forked_and_swapped_block_scaled_cache():
    """A partly filled tail block copied for a second writer, its rows of scales beside its codes, and swapped out and in."""
    Hq, Hkv, D, B, n, NB = 8, 2, 128, 16, 37, 12
    g = torch.Generator(device="cuda").manual_seed(2)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    kc, vc = (torch.full((NB, Hkv, B, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((NB, Hkv), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table, at = i32(7, 2, 9), torch.arange(n, device="cuda")
    api.pa_reshape_and_cache_scaled(kc, vc, ks, vs, draw(n, Hkv, D), draw(n, Hkv, D), table.long()[at // B] * B + at % B)
    api.pa_copy_blocks([kc], [vc], i32(9, 4).view(1, 2))           # the tail, for the second sample
    ks[4], vs[4] = ks[9], vs[9]
    both = torch.stack([table, i32(7, 2, 4)])
    x = draw(2, Hkv, D) * torch.tensor([1.0, 32.0], device="cuda").view(2, 1, 1)   # (the second's grows its block's scale)
    api.pa_reshape_and_cache_scaled(kc, vc, ks, vs, x.bfloat16(), x.bfloat16(), both[:, n // B].long() * B + n % B)

    def check(tables):
        p = Problem(1, Hq, Hkv, D, B, [n + 1] * 2, [1, 1], scaled=True)
        p.kc, p.vc, p.ks, p.vs, p.tables, p.q = (*(t.cpu().numpy() for t in (kc, vc, ks, vs, tables)), q)
        out = p.run()
        _check(p, out)
        return out

    q = torch.randn(2, Hq, D, generator=torch.Generator().manual_seed(3)).bfloat16()
    first = check(both)
    assert (ks[4] > ks[9]).all() and (vs[4] > vs[9]).all()
    out_k, out_v = (torch.empty(3, Hkv, B, D, dtype=torch.uint8).pin_memory() for _ in range(2))
    there, back = [[7, 0], [2, 1], [4, 2]], [[0, 1], [1, 3], [2, 5]]
    pairs = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    api.pa_swap_blocks([out_k], [out_v], [kc], [vc], pairs(there))
    held = [s[[7, 2, 4]].cpu() for s in (ks, vs)]
    kc[[2, 4]], vc[[2, 4]], ks[[2, 4]], vs[[2, 4]] = 0x7F, 0x7F, 255, 255
    api.pa_swap_blocks([kc], [vc], [out_k], [out_v], pairs(back))
    ks[[1, 3, 5]], vs[[1, 3, 5]] = (h.cuda() for h in held)
    both[1], both[0, 1] = i32(1, 3, 5), 3
    assert torch.equal(check(both), first)


@pytest.mark.parametrize("scaled", [False, True], ids=["bf16", "scaled"])
@pytest.mark.parametrize("S,new", [(1, 2), (1, 4), (1, 7), (1, 40), (24, 131)])
def test_keys_that_others_see_change_no_bit(scaled, S, new):
    """The even tokens' scores rise far above all before, at positions that the odd ones do not see."""
    p = Problem(14, 4, 1, 128, 16, [900] * S, [new] * S, "window", scaled=scaled)
    p.visible[:] = [0, 758]
    p.visible[::2] = [0, 900]
    if scaled:                                                     # (and theirs a little, in the tile of both)
        p.ks[p.tables[:, 752 // 16]] += 1
    else:
        p.kc[p.tables[:, 752 // 16], :, :6] += 0x80                # twice the values
    clean = p.run()
    for s in range(S):
        for j in range(758, 900, 7):
            p.kc[p.tables[s][j // 16], :, j % 16] = 0x7E if scaled else 0x4280      # 448, 2^6
    out = p.run()
    assert torch.equal(out[1::2], clean[1::2]) and not torch.equal(out[::2], clean[::2])
    _check(p, out, take=_few(12))
