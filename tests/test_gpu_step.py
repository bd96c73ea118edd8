"""pa_plan_step, pa_release_rows and pa_qk_norm_rope_cache against the oracle
(oracle/step.py), and a whole step of new tokens: planned, normed, rotated,
cached and attended to on the GPU.  Plans are whole numbers and must be
equal; projections carry one rounding."""
import math

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


class Plan:
    """Device state of a planner and the same state for the oracle."""

    def __init__(self, rows, max_blocks, pool, block, rng, status=True):
        self.B, self.NB, self.MB, self.R = block, pool, max_blocks, rows
        ids = [int(x) for x in rng.permutation(pool)]
        self.tables, self.blocks, self.lens = [[-1] * max_blocks for _ in range(rows)], [0] * rows, [0] * rows
        self.free = ids
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.d_tables = torch.tensor(self.tables, dtype=torch.int32, device="cuda")
        self.d_blocks = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.d_free = torch.tensor(ids, dtype=torch.int32, device="cuda")
        self.d_count = torch.tensor([len(ids)], dtype=torch.int32, device="cuda")

    def outputs(self, n_seqs, tokens):
        i = lambda *s: torch.full(s, 77, dtype=torch.int32, device="cuda")  # noqa: E731
        return i(n_seqs, self.MB), i(n_seqs), i(n_seqs + 1), i(tokens), i(tokens).long()

    def gpu(self, seq_rows, new, tokens, lens=None, free=True):
        d = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        out = self.outputs(len(seq_rows), tokens)
        api.pa_plan_step(*out, d(seq_rows), d(new), d(self.lens if lens is None else lens), self.d_tables, self.d_blocks,
                         self.d_free if free else None, self.d_count if free else None, self.B, self.NB,
                         status=self.status)
        return [x.cpu().tolist() for x in out]

    def check_state(self):
        assert self.d_blocks.cpu().tolist() == self.blocks
        n = int(self.d_count.item())
        assert n == len(self.free) and self.d_free.cpu().tolist()[:n] == self.free
        got = self.d_tables.cpu().tolist()
        for r in range(self.R):
            assert got[r][:self.blocks[r]] == self.tables[r][:self.blocks[r]]

    def step(self, seq_rows, new, pad=0):
        """Plan on both sides and compare everything; row_lens advance."""
        tokens = sum(n for r, n in zip(seq_rows, new) if r >= 0) + pad
        want = S.plan_step(seq_rows, new, self.lens, self.tables, self.blocks, self.free, self.B, tokens)
        got = self.gpu(seq_rows, new, tokens)
        assert self.status.item() == 0
        tables, ctx, start, positions, slots = want
        assert got[0] == [t + [-1] * (self.MB - len(t)) for t in tables]
        assert got[1:] == [ctx, start, positions, slots]
        self.check_state()
        for r, n in zip(seq_rows, new):
            if r >= 0:
                self.lens[r] += n


@pytest.mark.parametrize("block,max_blocks,seqs,seed", [(16, 8, 1, 0), (8, 33, 7, 1), (32, 20, 40, 2), (16, 64, 300, 3),
                                                        (8, 5, 1030, 4), (16, 3, 8192, 5)])
def test_steps_equal_the_oracle(block, max_blocks, seqs, seed):
    """Mixed batches (nothing cached, one token, chunks, none, padding among
    and after the requests), several steps on the same state."""
    rng = np.random.default_rng(seed)
    p = Plan(seqs + 5, max_blocks, (seqs + 5) * max_blocks, block, rng)
    room = max_blocks * block
    for _ in range(4):
        rows = [int(r) for r in rng.permutation(seqs + 5)[:seqs]]
        new = [int(min(rng.choice([0, 1, 1, 1, 2, block, 3 * block + 1]), room - p.lens[r])) for r in rows]
        for i in rng.integers(0, seqs, seqs // 6):
            rows[i] = -1
        p.step(rows, new, pad=int(rng.integers(0, 70)))


def test_a_long_chunk_and_an_empty_batch():
    rng = np.random.default_rng(6)
    p = Plan(3, 2048, 5000, 8, rng)
    p.step([2, 0], [16384, 1], pad=5)              # fills its row to the last position
    p.step([], [], pad=3)
    p.step([-1, -1], [4, 4], pad=0)                # padding brings nothing


def test_planning_again_takes_nothing_and_a_rejected_draft_keeps_its_blocks():
    rng = np.random.default_rng(7)
    p = Plan(4, 8, 24, 16, rng)
    p.step([1, 3], [16, 15])
    a = p.gpu([1, 3], [9, 9], 18)
    held = int(p.d_count.item())
    assert p.gpu([1, 3], [9, 9], 18) == a and int(p.d_count.item()) == held
    S.plan_step([1, 3], [9, 9], p.lens, p.tables, p.blocks, p.free, 16, 18)
    p.check_state()
    p.lens[1] += 2                                  # two of the nine were accepted
    p.lens[3] += 1
    p.step([3, 1], [3, 20])


def test_tables_reserved_by_the_host_manager():
    """Without a free list the rows' tables hold the blocks: the slots are the
    host manager's for the same positions."""
    alloc = api.BlockAllocator(40, 16)
    assert alloc.allocate(0, 100) == alloc.allocate(1, 33) == api.PA_OK
    rng = np.random.default_rng(8)
    p = Plan(2, 8, 40, 16, rng)
    tables, _ = alloc.build_tables([0, 1], 8)
    p.d_tables.copy_(torch.from_numpy(tables))
    p.d_blocks.copy_(torch.tensor([7, 3], dtype=torch.int32))
    got = p.gpu([1, 0], [3, 10], 13, lens=[90, 30], free=False)
    assert p.status.item() == 0
    assert got[4] == alloc.slot_mapping(1, 30, 3).tolist() + alloc.slot_mapping(0, 90, 10).tolist()
    assert got[0] == [tables[1].tolist(), tables[0].tolist()]
    p.gpu([1, 0], [19, 0], 19, lens=[90, 30], free=False)       # a fourth block, and none to take
    assert p.status.item() == api.PA_DEV_NO_BLOCKS


@pytest.mark.parametrize("rows,new,tokens,lens,bit", [
    ([0, 1], [40, 40], 80, None, "NO_BLOCKS"),           # one block short
    ([0, 4], [1, 1], 2, None, "BAD_ROW"),                # out of range
    ([2, 1, 2], [1, 1, 1], 3, None, "BAD_ROW"),          # the same row twice
    ([0, 1], [1, -1], 2, None, "BAD_CONTEXT"),
    ([0, 1], [1, 65], 66, None, "BAD_CONTEXT"),          # past the table
    ([0, 1], [3, 2], 4, None, "BAD_CONTEXT"),            # more than num_tokens
    ([0, 1], [1, 1], 2, [0, -3, 0, 0], "BAD_CONTEXT"),
    ([0, 1], [2147483647, 2147483647], 9, None, "BAD_CONTEXT"),
])
def test_a_refused_plan_changes_nothing(rows, new, tokens, lens, bit):
    rng = np.random.default_rng(9)
    p = Plan(4, 4, 7, 16, rng)
    p.step([3], [20])
    p.step([0], [1])                                     # four blocks left: 3 + 3 - 1 are needed
    got = p.gpu(rows, new, tokens, lens)
    assert p.status.item() == getattr(api, "PA_DEV_" + bit)
    assert got[2] == [0] * (len(rows) + 1)
    assert got[3] == [-1] * tokens and got[4] == [-1] * tokens
    p.check_state()


def test_a_free_count_out_of_range_is_refused():
    p = Plan(2, 4, 8, 16, np.random.default_rng(10))
    for n in (9, -1):
        p.d_count.fill_(n)
        p.status.zero_()
        p.gpu([0], [5], 5)
        assert p.status.item() == api.PA_DEV_NO_BLOCKS and p.d_count.item() == n
    assert p.d_blocks.cpu().tolist() == [0, 0]


def test_a_bad_block_id_gives_no_slot():
    p = Plan(2, 4, 8, 16, np.random.default_rng(11))
    p.d_free[-1] = 8                                     # outside the pool of 8
    p.d_free[-2] = -7
    got = p.gpu([0, 1], [3, 20], 23)
    assert p.status.item() == api.PA_DEV_BAD_BLOCK_ID
    assert got[4][:3] == [-1] * 3 and got[4][3:19] == [-1] * 16 and all(s >= 0 for s in got[4][19:])


def test_release_equals_the_oracle_and_refuses():
    rng = np.random.default_rng(12)
    p = Plan(30, 10, 250, 8, rng)
    p.step(list(range(30)), [int(n) for n in rng.integers(0, 60, 30)])
    rel = lambda rows: api.pa_release_rows(torch.tensor(rows, dtype=torch.int32, device="cuda"), p.d_tables,  # noqa: E731
                                           p.d_blocks, p.d_free, p.d_count, status=p.status)
    for rows in ([7, -1, 3], [29, 0, 1, 2], [7]):        # a row that holds nothing is fine
        rel(rows)
        S.release_rows(rows, p.tables, p.blocks, p.free)
        for r in rows:
            p.lens[r] = 0
        assert p.status.item() == 0
        p.check_state()
    p.step([7, 8], [31, 1])
    for rows, bit in (([5, 5], api.PA_DEV_BAD_ROW), ([30], api.PA_DEV_BAD_ROW)):
        p.status.zero_()
        rel(rows)
        assert p.status.item() == bit
        p.check_state()
    p.status.zero_()
    p.d_count.fill_(250)                                 # the list would overflow
    rel([6])
    assert p.status.item() == api.PA_DEV_BAD_CONTEXT and p.d_blocks[6].item() == p.blocks[6]


# ---------------------------------------------------------------------------
# norm + rotation + cache write
# ---------------------------------------------------------------------------

def _rope_case(T, Hq, Hkv, D, B, rot, norm, seed, longest=5000, packed=True):
    rng = np.random.default_rng(seed)
    if packed:
        qkv = I.bf16_normal((T, (Hq + 2 * Hkv) * D), seed).cuda()
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    else:
        q, k, v = (I.bf16_normal((T, h, D), seed + i).cuda() for i, h in enumerate((Hq, Hkv, Hkv)))
    NB = -(-T // B) + 3
    slots = rng.permutation(NB * B)[:T].astype(np.int64)
    pos = rng.integers(0, longest, T).astype(np.int32)
    pos[0] = longest - 1
    gains = [torch.from_numpy((1 + 0.2 * rng.standard_normal(D)).astype(np.float32)).cuda() for _ in range(2)] if norm \
        else [None, None]
    return q, k, v, pos, slots, gains, NB, api.rope_table(longest, rot)


def _expected(x, gain, eps, pos, rot, interleaved):
    """Exact rows and their tolerance before the final rounding, [T, H, D]:
    32-bit sums and products put a turned element within 2^-19 (|a| + |b|) of
    its pair (a, b): at most 19 additions and 8 products and factors in a row
    and the table's own rounding, each 2^-24, and rsqrt's two units."""
    x64 = A.bf16_to_f64(to_bits(x))
    y, tol = np.empty_like(x64), np.empty_like(x64)
    for t in range(x64.shape[0]):
        for h in range(x64.shape[1]):
            y[t, h] = S.norm_rope(x64[t, h], gain, eps, int(pos[t]), rot, interleaved)
            size = np.abs(S.norm_rope(x64[t, h], gain, eps, 0, rot, interleaved))
            pair = size.copy()
            c = np.arange(rot // 2)
            i, j = (2 * c, 2 * c + 1) if interleaved else (c, c + rot // 2)
            pair[i] = pair[j] = size[i] + size[j]
            tol[t, h] = pair * 2.0 ** -19
    return y, tol


def _close(got, want, tol, half_step, smallest=0.0):
    off = np.abs(got - want)
    assert (off <= tol + half_step * (np.abs(want) + tol) + smallest).all(), off.max()


@pytest.mark.parametrize("T,Hq,Hkv,D,B,rot,inter,norm,packed", [
    (1, 32, 8, 128, 16, 128, False, True, True),
    (37, 4, 2, 64, 8, 64, False, True, True),
    (19, 8, 1, 128, 32, 32, False, True, True),          # a quarter of each head turns
    (23, 2, 2, 64, 16, 16, True, True, False),
    (11, 16, 4, 128, 16, 128, True, False, True),
    (9, 6, 3, 64, 16, 48, False, False, False),
    (130, 1, 1, 128, 16, 112, True, True, True),
])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_norm_rope_cache_equals_the_oracle(T, Hq, Hkv, D, B, rot, inter, norm, packed, fp8):
    q, k, v, pos, slots, (qw, kw), NB, table = _rope_case(T, Hq, Hkv, D, B, rot, norm, 5 * T + Hq, packed=packed)
    scales = (np.float32(0.013), np.float32(0.021))
    if fp8:
        kc = torch.full((NB, Hkv, B, D), 0x5A, dtype=torch.uint8, device="cuda")
    else:
        kc = torch.full((NB, Hkv, B, D), 7.5, dtype=torch.bfloat16, device="cuda")
    vc, untouched = kc.clone(), kc.cpu().clone()
    out = torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    extra = dict(k_scale=float(scales[0]), v_scale=float(scales[1])) if fp8 else {}
    api.pa_qk_norm_rope_cache(out, kc, vc, q, k, v, torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda(), table,
                              q_weight=qw, k_weight=kw, eps=1e-5, interleaved=inter, status=st, **extra)
    assert st.item() == 0
    host = lambda w: None if w is None else w.double().cpu().numpy()  # noqa: E731
    want, tol = _expected(q, host(qw), 1e-5, pos, rot, inter)
    _close(A.bf16_to_f64(to_bits(out)), want, tol, 2.0 ** -8)
    want, tol = _expected(k, host(kw), 1e-5, pos, rot, inter)
    rows = lambda c: c.cpu().permute(0, 2, 1, 3).reshape(NB * B, Hkv, D)[torch.from_numpy(slots)]  # noqa: E731
    if fp8:
        s = float(scales[0])
        got = Q.e4m3_to_f64(rows(kc).numpy())
        want, tol = np.clip(want / s, -448, 448), tol / s + np.abs(want / s) * 2.0 ** -23
        _close(got, want, tol, 2.0 ** -4, 2.0 ** -10)    # below 2^-6 the codes are 2^-9 apart
        assert np.array_equal(rows(vc).numpy(), Q.quantize(v.float().cpu().numpy(), scales[1]))
    else:
        _close(A.bf16_to_f64(to_bits(rows(kc))), want, tol, 2.0 ** -8)
        assert np.array_equal(to_bits(rows(vc)), to_bits(v))
    # every other slot is as it was
    keep = np.setdiff1d(np.arange(NB * B), slots)
    flat = lambda c: c.cpu().permute(0, 2, 1, 3).reshape(NB * B, Hkv, D)[torch.from_numpy(keep)]  # noqa: E731
    for c in (kc, vc):
        assert torch.equal(flat(c).float() if not fp8 else flat(c), flat(untouched).float() if not fp8 else
                           flat(untouched))


def test_padding_bad_positions_and_bad_slots():
    T, Hq, Hkv, D, B = 8, 4, 2, 128, 16
    q, k, v, pos, slots, (qw, kw), NB, table = _rope_case(T, Hq, Hkv, D, B, 128, True, 3, longest=50)
    pos = np.array([4, -1, 49, 50, 7, 8, -5, 9], dtype=np.int32)
    slots = np.array([0, 1, 2, 3, -1, NB * B, 5, 6], dtype=np.int64)
    kc = torch.zeros((NB, Hkv, B, D), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    out = torch.full((T, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.pa_qk_norm_rope_cache(out, kc, vc, q, k, v, torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda(), table,
                              q_weight=qw, k_weight=kw, status=st)
    assert st.item() == api.PA_DEV_BAD_POSITION | api.PA_DEV_BAD_SLOT
    left = [bool((out[t] == 3.0).all()) for t in range(T)]
    assert left == [False, True, False, True, False, False, True, False]
    written = [bool((vc[s // B, :, s % B] != 0).any()) for s in range(8)]
    assert written == [True, False, True, False, False, False, True, False]
    assert (vc[1:] == 0).all()


def test_q_in_place_extreme_values_and_no_tokens():
    T, Hq, Hkv, D, B = 5, 8, 2, 64, 16
    q, k, v, pos, slots, (qw, kw), NB, table = _rope_case(T, Hq, Hkv, D, B, 64, True, 4, packed=False)
    q[0, 0] = 0.0                                            # a zero head stays zero: eps is inside the root
    q[1, 1] = 1e30                                           # squares beyond fp32: the mean is infinite
    kc = torch.zeros((NB, Hkv, B, D), dtype=torch.bfloat16, device="cuda")
    vc, p, s = kc.clone(), torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda()
    out = torch.empty_like(q)
    api.pa_qk_norm_rope_cache(out, kc, vc, q, k, v, p, s, table, q_weight=qw, k_weight=kw)
    assert (out[0, 0] == 0).all() and (out[1, 1] == 0).all()
    api.pa_qk_norm_rope_cache(q, kc, vc, q, k, v, p, s, table, q_weight=qw, k_weight=kw)
    assert torch.equal(out.view(torch.int16), q.view(torch.int16))
    api.pa_qk_norm_rope_cache(out[:0], kc, vc, q[:0], k[:0], v[:0], p[:0], s[:0], table)
    with pytest.raises(ValueError, match="contiguous"):
        api.pa_qk_norm_rope_cache(out[:, :4], kc, vc, q[:, ::2], k, v, p, s, table)


# ---------------------------------------------------------------------------
# a whole step
# ---------------------------------------------------------------------------

def _random_tree(n, rng):
    seen = []
    for i in range(n):
        up = int(rng.integers(0, i)) if i else -1
        seen.append((seen[up] if up >= 0 else 0) | 1 << i)
    return seen


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_steps_of_new_tokens_from_projections_to_attention(fp8):
    """Prompt chunks, then drafts verified under a tree mask of which a part is
    kept, then single tokens: each step planned, normed, rotated, cached and
    attended to on the GPU alone, captured as a graph and replayed, and
    compared with the oracle over the cache as the GPU left it."""
    Hq, Hkv, D, B, R, MB = 8, 2, 128, 16, 4, 6
    rng = np.random.default_rng(20)
    NB, T, scale, dev = R * MB, 64, 1 / math.sqrt(D), "cuda"
    p = Plan(R, MB, NB, B, rng)
    cache = lambda: (torch.full((NB, Hkv, B, D), 0x7F, dtype=torch.uint8, device=dev) if fp8 else  # noqa: E731
                     I.nan_pool((NB, Hkv, B, D), dev))
    kc, vc = cache(), cache()
    table = api.rope_table(MB * B, D)
    scales = dict(k_scale=0.02, v_scale=0.02) if fp8 else {}
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
    rows, new, lens = i32(R), i32(R), i32(R)
    tables, ctx, start, pos = i32(R, MB), i32(R), i32(R + 1), i32(T)
    slots, mask = torch.zeros(T, dtype=torch.int64, device=dev), torch.zeros(T, dtype=torch.int64, device=dev)
    qkv = torch.zeros(T, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16, device=dev)
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    q_rot = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=dev)
    out = torch.zeros(T, Hq, D, dtype=torch.float32, device=dev)
    ws = api.decode_multi_workspace(40, Hq, Hkv, D)
    st = torch.zeros(1, dtype=torch.int32, device=dev)

    def step():
        api.pa_plan_step(tables, ctx, start, pos, slots, rows, new, lens, p.d_tables, p.d_blocks, p.d_free, p.d_count, B,
                         NB, status=st)
        api.pa_qk_norm_rope_cache(q_rot, kc, vc, q, k, v, pos, slots, table, status=st, **scales)
        api.pa_decode_multi(out, q_rot, kc, vc, tables, start, ctx, 40, B, scale, Hq, Hkv, D, MB * B, tree_mask=mask,
                            workspace=ws, status=st, **scales)

    # captured once, on a batch that brings nothing
    rows.fill_(-1)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n_step, (batch, bring) in enumerate([([2, 0, 3, -1], [40, 1, 17, 0]), ([0, 2, -1, 3], [5, 9, 0, 16]),
                                             ([3, 2, 1, 0], [1, 1, 1, 1])]):
        words, total = [], 0
        for r, n in zip(batch, bring):
            words += _random_tree(n, rng) if n_step else [(2 << i) - 1 for i in range(n)]
            total += n
        rows.copy_(torch.tensor(batch))
        new.copy_(torch.tensor(bring))
        lens.copy_(torch.tensor(p.lens))
        mask[:total] = torch.tensor(words)
        qkv[:] = I.bf16_normal(tuple(qkv.shape), 30 + n_step).to(dev)
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert st.item() == 0
        want = S.plan_step(batch, bring, p.lens, p.tables, p.blocks, p.free, B, T)
        assert pos.cpu().tolist() == want[3] and slots.cpu().tolist() == want[4]
        p.check_state()
        kd = Q.dequantize(kc.cpu().numpy(), 0.02) if fp8 else to_bits(kc)
        vd = Q.dequantize(vc.cpu().numpy(), 0.02) if fp8 else to_bits(vc)
        ref = A.paged_multi(to_bits(q_rot), kd, vd, tables.cpu().numpy(), want[2], want[1], scale, B, words)
        got = out.cpu().double().numpy()
        assert np.abs(got[:total] - ref[:total]).max() <= 2e-3
        assert (got[total:] == 9.0).all()                     # rows behind the last token
        for r, n in zip(batch, bring):
            if r >= 0:
                p.lens[r] += n if n_step != 1 else (n + 1) // 2   # half of a draft is kept


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("Hq,Hkv,D,rot,inter,norm", [(32, 8, 128, 128, False, True), (17, 3, 64, 48, True, True),
                                                     (13, 2, 128, 64, False, False)])
def test_many_tokens_equal_the_same_tokens_a_few_at_a_time(Hq, Hkv, D, rot, inter, norm, fp8):
    """The path that large calls take, with padding and bad places among its
    tokens, gives the bits of the small calls' (which the oracle checks)."""
    T, B = 12000000 // ((Hq + 2 * Hkv) * D) + 3, 16
    q, k, v, pos, slots, (qw, kw), NB, table = _rope_case(T, Hq, Hkv, D, B, rot, norm, 50, longest=900)
    pos[5], pos[6], pos[T - 1] = -1, 900, 17
    slots[7], slots[8] = -1, NB * B
    pos, slots = torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda()
    extra = dict(k_scale=0.013, v_scale=0.021) if fp8 else {}
    dt = torch.uint8 if fp8 else torch.bfloat16
    got = []
    for step in (T, 1000):
        kc = torch.zeros((NB, Hkv, B, D), dtype=dt, device="cuda")
        vc, out = kc.clone(), torch.zeros((T, Hq, D), dtype=torch.bfloat16, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        for i in range(0, T, step):
            part = slice(i, min(T, i + step))
            api.pa_qk_norm_rope_cache(out[part], kc, vc, q[part], k[part], v[part], pos[part], slots[part], table,
                                      q_weight=qw, k_weight=kw, interleaved=inter, status=st, **extra)
        assert st.item() == api.PA_DEV_BAD_POSITION | api.PA_DEV_BAD_SLOT
        got.append((out, kc, vc))
    for a, b in zip(*got):
        a, b = (x.view(torch.int16) if x.dtype == torch.bfloat16 else x for x in (a, b))
        assert torch.equal(a, b)
    assert (got[0][0][5] == 0).all() and (got[0][0][6] == 0).all() and (got[0][0][7] != 0).any()


@pytest.mark.parametrize("seqs,max_blocks,rows", [
    (2, 8, 3),                       # one cluster
    (4, 1 << 17, 5),                 # two launches: tables past what the cluster takes
])
@pytest.mark.parametrize("bad", ["blocks", "row"])
def test_a_refused_plan_with_less_blocks_than_its_lengths_need(seqs, max_blocks, rows, bad):
    """Rows that hold fewer blocks than their positions fill (they would take
    the rest): a refused step shows what the rows have and takes nothing."""
    p = Plan(rows, max_blocks, 9, 16, np.random.default_rng(13))
    p.d_tables.fill_(-1)
    lens = [100] + [0] * (rows - 1)
    if bad == "blocks":
        p.d_count.fill_(3)
    seq_rows = [0, 1 if bad == "blocks" else rows] + [-1] * (seqs - 2)
    before = p.d_tables.clone(), p.d_blocks.clone(), p.d_count.clone()
    got = p.gpu(seq_rows, [20, 1] + [0] * (seqs - 2), 30, lens)
    assert p.status.item() == (api.PA_DEV_NO_BLOCKS if bad == "blocks" else api.PA_DEV_BAD_ROW)
    assert got[1][0] == 100 and got[2] == [0] * (seqs + 1) and got[3] == [-1] * 30 and got[4] == [-1] * 30
    assert all(x == -1 for t in got[0] for x in t)
    for a, b in zip(before, (p.d_tables, p.d_blocks, p.d_count)):
        assert torch.equal(a, b)
    p.d_count.fill_(9)
    p.status.zero_()
    if bad == "blocks":                                  # enough of them: the rest of the row's is taken with the step's
        got = p.gpu(seq_rows, [20, 1] + [0] * (seqs - 2), 30, lens)
        assert p.status.item() == 0 and p.d_blocks.cpu().tolist()[:2] == [8, 1] and p.d_count.item() == 0
        assert got[0][0][:8] == p.free[:0:-1] and got[0][1][0] == p.free[0]
        assert got[3][:21] == list(range(100, 120)) + [0]


@pytest.mark.parametrize("seqs,max_blocks,rows,tokens", [
    (2048, 4, 2050, 0), (2049, 4, 2050, 0),              # the most requests of one cluster, and one more
    (100, 2000, 101, 8750), (100, 2000, 101, 8751),      # its most table entries and tokens
    (3, 4, 262144, 5),                                   # the most rows
])
def test_steps_at_the_bounds_of_the_single_launch(seqs, max_blocks, rows, tokens):
    rng = np.random.default_rng(14)
    p = Plan(rows, max_blocks, 5000, 8, rng)
    which = [int(r) for r in rng.permutation(rows)[:seqs]]
    for _ in range(2):
        new = [int(n) for n in rng.integers(0, 3, seqs)]
        p.step(which, new, pad=max(0, tokens - sum(new)))
        p.step(which, [0] * (seqs - 1) + [1], pad=tokens)


def test_plans_of_two_pools_at_once_and_replayed():
    """Two planners on two streams, and both captured: each keeps to its own
    state."""
    rng = np.random.default_rng(15)
    plans = [Plan(40, 64, 900, 16, rng) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in plans]
    d = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    news = [[int(n) for n in rng.integers(0, 4, 40)] for _ in plans]
    outs = [p.outputs(40, 130) for p in plans]
    args = [(d(list(range(40))), d(n), d([0] * 40)) for n in news]
    run = lambda i: api.pa_plan_step(*outs[i], *args[i], plans[i].d_tables, plans[i].d_blocks, plans[i].d_free,  # noqa: E731
                                     plans[i].d_count, 16, 900, status=plans[i].status)
    lens = [a[2] for a in args]
    torch.cuda.synchronize()
    for step in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                run(i)
                lens[i].add_(args[i][1])
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(i)
            lens[i].add_(args[i][1])
        graphs.append(g)
    for step in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for p, n, o in zip(plans, news, outs):
        for step in range(9):
            want = S.plan_step(list(range(40)), n, p.lens, p.tables, p.blocks, p.free, 16, 130)
            p.lens = [a + b for a, b in zip(p.lens, n)]
        assert p.status.item() == 0
        p.check_state()
        assert [x.cpu().tolist() for x in o[1:]] == list(want[1:])


def test_tensors_of_wrong_type_shape_place_or_layout_are_refused():
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    b = lambda *s: z(*s, dt=torch.bfloat16)  # noqa: E731
    plan = dict(block_tables=z(2, 4), context_lens=z(2), query_start=z(3), positions=z(5), slot_mapping=z(5).long(),
                seq_rows=z(2), new_lens=z(2), row_lens=z(8), row_tables=z(8, 4), row_blocks=z(8), free_blocks=z(64),
                free_count=z(1), block_size=16, num_blocks=64)
    rope = dict(q_out=b(3, 4, 64), k_cache=b(2, 2, 16, 64), v_cache=b(2, 2, 16, 64), q=b(3, 4, 64), k=b(3, 2, 64),
                v=b(3, 2, 64), positions=z(3), slot_mapping=z(3).long(), cos_sin=z(9, 64, dt=torch.float32))
    multi = dict(out=b(3, 4, 64), q=b(3, 4, 64), k_cache=b(2, 2, 16, 64), v_cache=b(2, 2, 16, 64), block_tables=z(1, 2),
                 query_start=z(2), context_lens=z(1), max_query_len=3, block_size=16, scale=0.125, n_q_heads=4,
                 n_kv_heads=2, d_head=64, max_context_len=32)
    for fn, good, cases in (
            (api.pa_plan_step, plan, [
                (dict(context_lens=z(3)), ValueError, "context_lens must be"), (dict(positions=z(6)), ValueError, "slot_mapping must be"),
                (dict(row_tables=z(4, 8).t()), ValueError, "row_tables must be contiguous"),
                (dict(new_lens=z(2).cpu()), ValueError, "new_lens must be a CUDA tensor"),
                (dict(row_blocks=z(8).long()), TypeError, "row_blocks must be torch.int32"),
                (dict(free_count=z(2)), ValueError, "free_count must be"), (dict(seq_rows=None), TypeError, "seq_rows must be a torch"),
                (dict(block_size=1 << 40), ValueError, "outside 32 bits"), (dict(block_size="16"), TypeError, None)]),
            (api.pa_qk_norm_rope_cache, rope, [
                (dict(q=b(3, 64, 4).transpose(1, 2)), ValueError, "q must have the heads"),
                (dict(k=b(3, 4, 64)), ValueError, "k must be"), (dict(v=b(4, 2, 64)), ValueError, "v must be"),
                (dict(cos_sin=z(9, 64)), TypeError, "cos_sin must be torch.float32"),
                (dict(q_out=b(6, 4, 64)[::2]), ValueError, "q_out must be contiguous"),
                (dict(k_scale=0.1, v_scale=0.1), TypeError, "k_cache must be torch.uint8"),
                (dict(q_weight=z(63, dt=torch.float32), k_weight=z(64, dt=torch.float32)), ValueError, "q_weight must be")]),
            (api.pa_decode_multi, multi, [
                (dict(out=z(3, 4, 64)), TypeError, "out must be bfloat16"), (dict(q=b(3, 2, 64)), ValueError, "q must be"),
                (dict(v_cache=b(2, 2, 8, 64)), ValueError, "v_cache must be"), (dict(query_start=z(1)), ValueError, "query_start must be"),
                (dict(tree_mask=z(2).long()), ValueError, "tree_mask must be"), (dict(k_scale=0.1), ValueError, "go together"),
                (dict(workspace=z(16)), TypeError, "workspace must be torch.uint8"), (dict(scale="x"), TypeError, None)])):
        assert fn(**good) == api.PA_OK
        for change, error, text in cases:
            with pytest.raises(error, match=text):
                fn(**dict(good, **change))
    torch.cuda.synchronize()


@pytest.mark.parametrize("max_blocks", [8, 1 << 17], ids=["one cluster", "two launches"])
@pytest.mark.parametrize("rows,new,held,bit", [
    ([2, 1, 2, 0], [1, 1, 4, 1], None, "BAD_ROW"),       # the same row twice, with different lengths
    ([2, 2, 2, 2], [0, 0, 0, 0], None, "BAD_ROW"),
    ([1, 2, 0, -1], [-1, 1, 2, 5], None, "BAD_CONTEXT"),
    ([1, 2, 0, 7], [2147483647, 1, 2, 5], None, "BAD_CONTEXT|BAD_ROW"),
    ([1, 2, 0, -1], [1, 1, 1, 1], -1, "BAD_CONTEXT"),    # a row that holds fewer blocks than none
    ([1, 2, 0, -1], [1, 1, 1, 1], 1 << 30, "BAD_CONTEXT"),
])
def test_a_refused_plan_shows_what_every_named_row_has(max_blocks, rows, new, held, bit):
    """Every n is 0, of the entries that are at fault as well, and of both that name one row whichever comes first."""
    p = Plan(5, max_blocks, 30, 8, np.random.default_rng(16))
    p.step([2, 0, 1], [20, 7, 33])
    if held is not None:
        p.d_blocks[1] = held
    before = p.d_tables.clone(), p.d_blocks.clone(), p.d_count.clone()
    want = 0
    for name in bit.split("|"):
        want |= getattr(api, "PA_DEV_" + name)
    for _ in range(20):
        p.status.zero_()
        got = p.gpu(rows, new, 12)
        assert p.status.item() == want
        there = [r if 0 <= r < 5 else None for r in rows]
        assert got[1] == [0 if r is None else p.lens[r] for r in there]
        for t, r in zip(got[0], there):
            nb = 0 if r is None else -(-p.lens[r] // 8)
            assert t[:nb] == p.tables[r][:nb] if nb else True
            assert all(x == -1 for x in t[nb:])
        assert got[2] == [0] * 5 and got[3] == [-1] * 12 and got[4] == [-1] * 12
    for a, b in zip(before, (p.d_tables, p.d_blocks, p.d_count)):
        assert torch.equal(a, b)


def test_the_readmes_example_runs_over_a_state_that_holds_together():
    """The steps planned on the GPU keep to blocks of their own, attend to positions that they have written, and give
    what the oracle gives over the cache as it is left."""
    import os
    import re
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    with open(path) as f:
        (code,) = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    x = {}
    exec(compile(code, "README.md", "exec"), x)
    torch.cuda.synchronize()
    B, NB, ctx, tables = x["B"], x["NB"], x["context_lens"].tolist(), x["block_tables"].cpu().numpy()
    owned = set(x["alloc"].free_list())
    assert ctx == [1004, 44] and x["row_lens"].tolist() == [1002, 44] and x["row_blocks"].tolist() == [0, 0]
    assert sorted(x["free_blocks"].tolist()) == sorted(set(range(NB)) - owned) and x["free_count"].item() == NB - len(owned)
    for t, c in zip(tables, ctx):
        ids = t[:-(-c // B)]
        assert not owned & set(ids.tolist())
        slots = torch.from_numpy(ids[np.arange(c) // B]).long().cuda(), torch.from_numpy(np.arange(c) % B).cuda()
        for cache in (x["k_cache"], x["v_cache"]):
            assert (cache[slots[0], :, slots[1]] != 0).any(-1).all()
    want = A.paged_multi(to_bits(x["q_out"]), to_bits(x["k_cache"]), to_bits(x["v_cache"]), tables,
                         x["query_start"].tolist(), ctx, x["scale"], B)
    off = np.abs(x["out"].double().cpu().numpy() - want)
    assert (off <= 2.0 ** -8 * np.abs(want) + 2e-3).all()
