"""The oracle of the router's choice by scores: worked rows, and its gradient
against differences (no GPU)."""
import numpy as np
import pytest

from oracle import select as S


def test_a_worked_row():
    z = [[np.log(1.0), np.log(3.0), np.log(2.0), np.log(2.0)]]
    idx, w = S.router_select(z, 2)
    assert idx.tolist() == [[1, 2]] and np.allclose(w, [[0.6, 0.4]])
    idx, w = S.router_select(z, 2, renorm=False, scale=2.0)
    assert idx.tolist() == [[1, 2]] and np.allclose(w, [[2 * 3 / 8, 2 * 2 / 8]])
    # the bias moves the choice, not the weight
    idx, w = S.router_select(z, 1, bias=[1.0, 0, 0, 0], renorm=False)
    assert idx.tolist() == [[0]] and np.allclose(w, [[1 / 8]])
    # sigmoid(log x) = x / (1 + x)
    idx, w = S.router_select(z, 4, score="sigmoid", renorm=False)
    assert idx.tolist() == [[1, 2, 3, 0]] and np.allclose(w, [[0.75, 2 / 3, 2 / 3, 0.5]])


def test_groups():
    z = [[0.0, 5.0, 3.0, 3.0, 4.0, 0.0]]
    assert S.router_select(z, 2, groups=3, top_groups=1)[0].tolist() == [[1, 0]]              # by the largest
    s = 1 / (1 + np.exp(-np.array(z[0])))
    assert s[2] + s[3] > s[0] + s[1]
    assert S.router_select(z, 2, "sigmoid", groups=3, top_groups=1, best=2)[0].tolist() == [[2, 3]]
    assert S.router_select(z, 2, "sigmoid", groups=3, top_groups=2, best=2)[0].tolist() == [[1, 2]]


def test_masked_experts_take_no_part():
    low = -3.4e38
    z = [[low, 1.0, -np.inf, np.nan], [low, low, -np.inf, np.nan], [np.inf, 1.0, np.inf, 0.0]]
    idx, w = S.router_select(z, 2)
    assert idx.tolist() == [[1, -1], [-1, -1], [0, 2]]
    assert w.tolist() == [[1, 0], [0, 0], [0.5, 0.5]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(score, renorm):
    r = np.random.RandomState(3)
    z, dw = r.randn(4, 9), r.randn(4, 3)
    idx, w = S.router_select(z, 3, score, renorm=renorm, scale=1.7)
    got = S.router_select_bwd(z, idx, dw, score, renorm, 1.7)

    def f(x):
        out = 0.0
        for t in range(4):
            s = S._row_scores(x[t], score)[idx[t]]
            out += (1.7 * (s / s.sum() if renorm else s) * dw[t]).sum()
        return out

    h = 1e-6
    for t in range(4):
        for e in range(9):
            d = np.zeros_like(z)
            d[t, e] = h
            # central differences: h^2 of the third derivative, and 64 bits' 1e-16 / h
            assert abs((f(z + d) - f(z - d)) / (2 * h) - got[t, e]) < 1e-8
