"""Pins of the router oracle: its choice against an exhaustive ranking, its gates against
the definition, its gradient against differences."""
import numpy as np
import pytest

from oracle import route as RT


def test_plain_softmax_choice_and_gates():
    l = np.array([[0.0, 2.0, 2.0, -1.0]])
    ids, gates = RT.route(l, None, 2)
    assert ids.tolist() == [[1, 2]] and np.allclose(gates, [[0.5, 0.5]])
    ids, gates = RT.route(l, None, 2, renorm=False, scale=2.0)
    p = np.exp(l) / np.exp(l).sum()
    assert np.allclose(gates, 2.0 * p[:, [1, 2]])


def test_bias_moves_the_choice_but_not_the_gates():
    l = np.array([[1.0, 0.5, 0.0]])
    b = np.array([0.0, 0.0, 5.0])
    ids, gates = RT.route(l, b, 2, score="sigmoid", renorm=False)
    assert ids.tolist() == [[2, 0]]
    assert np.allclose(gates, 1 / (1 + np.exp(-l[:, [2, 0]])))


def test_groups_by_the_sum_of_two():
    # group 0 holds the best expert, group 1 the best pair
    l = np.array([[3.0, -9.0, 2.0, 2.0]])
    assert RT.route(l, None, 1, score="sigmoid", groups=2, top_groups=1, group_top=1)[0][0, 0] == 0
    assert RT.route(l, None, 1, score="sigmoid", groups=2, top_groups=1, group_top=2)[0][0, 0] == 2


def test_masked_experts_fill_up_with_gate_zero():
    l = np.array([[-np.inf, 1.0, -np.inf, -np.inf], [-np.inf] * 4])
    ids, gates = RT.route(l, None, 3)
    assert ids.tolist() == [[1, 0, 2], [0, 1, 2]]
    assert gates.tolist() == [[1.0, 0.0, 0.0], [0.0, 0.0, 0.0]]


def test_low_sigmoid_logits_keep_their_ratio():
    l = np.array([[-1000.0, -1000.0 + np.log(3.0)]])
    _, gates = RT.route(l, None, 2, score="sigmoid")
    assert np.allclose(gates, [[0.75, 0.25]])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(1)
    l = rng.standard_normal((3, 7))
    bias = 0.1 * rng.standard_normal(7)
    bias[2] = -np.inf
    dg = rng.standard_normal((3, 3))
    kw = dict(score=score, renorm=renorm, scale=1.5)
    ids, gates = RT.route(l, bias, 3, **kw)
    got = RT.route_backward(l, bias, ids, gates, dg, **kw)
    h = 1e-6
    for g in range(3):
        for e in range(7):
            up, dn = l.copy(), l.copy()
            up[g, e] += h
            dn[g, e] -= h
            f = []
            for x in (up, dn):
                i, v = RT.route(x, bias, 3, **kw)
                assert np.array_equal(i, ids)
                f.append((v * dg).sum())
            assert abs((f[0] - f[1]) / (2 * h) - got[g, e]) < 1e-7
