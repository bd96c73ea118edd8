"""The oracle of a step's plan, norm and rotation, and tree attention, pinned
by closed forms, invariants and the reference block manager.  CPU only."""
import math

import numpy as np
import pytest

from oracle import allocator as AL
from oracle import attention as A
from oracle import step as S


def test_plan_equals_the_block_managers_steps():
    """Prompts admitted and extended position by position by the reference
    block manager, and the same requests planned from their lengths, hold the
    same blocks at the same slots."""
    rng = np.random.default_rng(0)
    B, NB, MB = 4, 64, 12
    ref = AL.RefAllocator(NB, B)
    tables, blocks, lens = [[-1] * MB for _ in range(5)], [0] * 5, [0] * 5
    free = list(reversed(range(NB)))                       # a fresh manager hands out 0, 1, 2, ...
    first = [int(n) for n in rng.integers(1, 15, 5)]
    got = S.plan_step(range(5), first, lens, tables, blocks, free, B, sum(first))
    for s, n in enumerate(first):
        ref.allocate(s, n)
        lens[s] = n
    for s in range(5):
        assert tables[s][:blocks[s]] == ref.block_tables[s]
    for _ in range(20):
        order = [int(x) for x in rng.permutation(5)]
        got = S.plan_step(order, [1] * 5, lens, tables, blocks, free, B, 7)
        slots = [ref.append_slot(s)[1] for s in order]
        assert got[4] == slots + [-1, -1] and got[3] == [lens[s] for s in order] + [-1, -1]
        assert got[2] == list(range(6)) and got[1] == [lens[s] + 1 for s in order]
        for s in order:
            lens[s] += 1
            assert tables[s][:blocks[s]] == ref.block_tables[s]
    S.release_rows([3, -1, 1], tables, blocks, free)
    ref.free(3)
    ref.free(1)
    assert free == ref.free_blocks and blocks[3] == blocks[1] == 0


def test_plan_changes_nothing_when_blocks_run_out():
    tables, blocks, free = [[-1] * 4, [-1] * 4], [0, 0], [5]
    assert S.plan_step([0, 1], [3, 3], [0, 0], tables, blocks, free, 4, 6) is None
    assert tables == [[-1] * 4, [-1] * 4] and blocks == [0, 0] and free == [5]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_depends_on_distance_alone(interleaved):
    rng = np.random.default_rng(1)
    q, k = rng.normal(size=(2, 32))
    turn = lambda x, p: S.norm_rope(x, None, 0.0, p, 32, interleaved)  # noqa: E731
    assert np.isclose(np.linalg.norm(turn(q, 1234)), np.linalg.norm(q))
    np.testing.assert_allclose(turn(q, 0), q)
    np.testing.assert_allclose(turn(q, 17) @ turn(k, 5), turn(q, 112) @ turn(k, 100))


def test_rotation_by_hand_and_partial():
    x = np.arange(1.0, 7.0)
    y = S.norm_rope(x, None, 0.0, 2, 4, False, base=100.0)
    a0, a1 = 2.0, 2.0 * 0.1
    want = [x[0] * math.cos(a0) - x[2] * math.sin(a0), x[1] * math.cos(a1) - x[3] * math.sin(a1),
            x[2] * math.cos(a0) + x[0] * math.sin(a0), x[3] * math.cos(a1) + x[1] * math.sin(a1), 5.0, 6.0]
    np.testing.assert_allclose(y, want)
    z = S.norm_rope(x, None, 0.0, 2, 4, True, base=100.0)
    np.testing.assert_allclose(z[:2], [math.cos(a0) - 2 * math.sin(a0), 2 * math.cos(a0) + math.sin(a0)])


def test_norm_by_hand():
    y = S.norm_rope(np.array([3.0, 4.0]), [2.0, 1.0], 0.5, 0, 2, False)
    np.testing.assert_allclose(y, np.array([6.0, 4.0]) / math.sqrt(13.0))


def test_tree_attention_of_a_chain_is_causal_and_of_a_leaf_is_its_path():
    rng = np.random.default_rng(2)
    Hkv, Hq, D, B, n, C = 2, 4, 8, 4, 4, 11
    k, v = rng.normal(size=(2, 5, Hkv, B, D))
    tab, start, ctx = np.array([[4, 0, 2]]), [0, n], [C]
    q = rng.normal(size=(n, Hq, D))
    chain = [(2 << i) - 1 for i in range(n)]
    np.testing.assert_allclose(A.paged_multi(q, k, v, tab, start, ctx, 0.3, B, chain),
                               A.paged_prefill(q, k, v, tab, start, ctx, 0.3, B))
    # token 3 follows token 1 follows the context: the same as a causal row whose cache leaves tokens 0 and 2 out
    K, V = A.gather_kv(k, v, tab[0], C, B)
    keep = list(range(C - n)) + [C - n + 1, C - n + 3]
    got = A.paged_multi(q, k, v, tab, start, ctx, 0.3, B, [1, 2, 4, 0b1010 | 1 << 60])
    for g in range(Hq):
        want = A.softmax_attention(q[3, g], K[g // 2][keep], V[g // 2][keep], 0.3)
        np.testing.assert_allclose(got[3, g], want)
    # nothing cached and an empty word: nothing to see
    got = A.paged_multi(q, k, v, tab, start, [n], 0.3, B, [0, 1, 1, 0])
    assert (got[0] == 0).all() and (got[3] == 0).all() and (got[1] != 0).any()
