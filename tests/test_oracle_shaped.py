"""Pins of the oracle's shaped attention, its block-scaled codes and its
rotation by several axes.  CPU only."""
import math

import numpy as np
import pytest

from oracle import attention as A
from oracle import quant as Q
from oracle import step as S


def _pool(seed=0, ctxs=(5, 23, 40), B=8, Hkv=2, D=4):
    rng = np.random.default_rng(seed)
    nb = [-(-c // B) for c in ctxs]
    tables, at = np.full((len(ctxs), max(nb)), -1), 0
    ids = rng.permutation(sum(nb) + 2)
    for s, n in enumerate(nb):
        tables[s, :n] = ids[at:at + n]
        at += n
    kc, vc = rng.standard_normal((2, sum(nb) + 2, Hkv, B, D))
    return rng, kc, vc, tables


def test_without_a_shape_it_is_the_prefill():
    rng, kc, vc, tables = _pool()
    q = rng.standard_normal((9, 4, 4))
    args = (q, kc, vc, tables, [0, 2, 3, 9], [5, 23, 40], 0.7, 8)
    assert np.allclose(A.paged_shaped(*args), A.paged_prefill(*args), rtol=1e-12, atol=0)


def test_a_window_is_the_attention_of_its_positions():
    rng, kc, vc, tables = _pool()
    q = rng.standard_normal((1, 4, 4))
    out = A.paged_shaped(q, kc, vc, tables[2:], [0, 1], [40], 0.7, 8, [[11, 30]])
    K, V = A.gather_kv(kc, vc, tables[2], 40, 8)
    for g in range(4):
        assert np.allclose(out[0, g], A.softmax_attention(q[0, g], K[g // 2][11:30], V[g // 2][11:30], 0.7), rtol=1e-12)
    assert (A.paged_shaped(q, kc, vc, tables[2:], [0, 1], [40], 0.7, 8, [[7, 7]]) == 0).all()
    clipped = A.paged_shaped(q, kc, vc, tables[2:], [0, 1], [40], 0.7, 8, [[-3, 900]])
    assert np.allclose(clipped, A.paged_decode(q, kc, vc, tables[2:], [40], 0.7, 8), rtol=1e-12)


def test_closed_forms_of_cap_and_bias():
    # equal keys of score 2: any cap leaves equal weights; a bias by distance a geometric series
    K = np.ones((3, 1))
    s = A.shaped_scores([2.0], K, 1.0, 2, softcap=0.5)
    assert np.allclose(s, 0.5 * math.tanh(4.0))
    assert np.allclose(A.shaped_scores([2.0], K, 1.0, 2, slope=math.log(2)), 2 - np.log([4, 2, 1]))
    assert np.allclose(A.shaped_scores([2.0], K, 1.0, 0, slope=1.0), [2, 1, 0])          # ahead of the token too
    assert np.allclose(A.shaped_scores([2.0], K, 1.0, 2, softcap=1e9), 2)                # a cap far away caps nothing
    # two positions, the cap before the bias
    got = A.shaped_scores([1.0], np.array([[3.0], [-3.0]]), 1.0, 1, softcap=1.0, slope=0.25)
    assert np.allclose(got, [math.tanh(3) - 0.25, -math.tanh(3)])


@pytest.mark.parametrize("top,e", [(448.0, 0), (448.1, 1), (224.0, -1), (1.75, -8), (1.76, -7), (1.0, -8), (0.0, -127)])
def test_the_least_exponent(top, e):
    assert Q.least_exponent(top) == e


def test_append_scaled_by_hand():
    codes, scales = np.zeros((2, 1, 4, 1), np.uint8), np.zeros((2, 1), np.uint8)
    code = lambda v: int(Q.f64_to_e4m3(v))  # noqa: E731
    x = np.array([448.0, 7.0]).reshape(2, 1, 1)
    Q.append_scaled(codes, scales, x, [4, 5], 4)                  # a block from its offset 0 on: 2^0
    assert scales[1, 0] == 127 and codes[1, 0, :2, 0].tolist() == [code(448), code(7)]
    Q.append_scaled(codes, scales, np.array([[[1.0]]]), [6], 4)   # smaller: the scale stays
    assert scales[1, 0] == 127 and codes[1, 0, 2, 0] == code(1)
    Q.append_scaled(codes, scales, np.array([[[1792.0]]]), [7], 4)   # 4 * 448: all codes a quarter
    assert scales[1, 0] == 129 and codes[1, 0, :, 0].tolist() == [code(112), code(1.75), code(0.25), code(448)]
    assert np.allclose(Q.dequantize_scaled(codes, scales)[1, 0, :, 0], [448, 7, 1, 1792])
    Q.append_scaled(codes, scales, np.array([[[0.5]]]), [4], 4)   # begun anew
    assert scales[1, 0] == 118 and codes[1, 0, 0, 0] == code(256.0)
    assert (codes[0] == 0).all() and scales[0, 0] == 0


def test_several_axes_turn_each_pair_by_its_own():
    x = np.arange(1.0, 9.0)
    got = S.norm_rope(x, None, 0.0, [3, 5, 7, 0], 8, False)
    for c, p in enumerate([3, 5, 7, 0]):
        one = S.norm_rope(x, None, 0.0, p, 8, False)
        assert got[c] == one[c] and got[c + 4] == one[c + 4]
    assert got[3] == x[3]
