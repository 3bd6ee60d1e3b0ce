"""The router's choice by scores and its gradient against the float64 oracle
(moe_router_select, moe_router_select_bwd)."""
import itertools

import numpy as np
import pytest
import torch

import dropless_grouped_gemm_gb300 as M
from oracle import select as S

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16
DEV = "cuda"


def _logits(T, E, dt, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn((T, E), generator=g)).to(dt)


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _check(z, k, bias=None, **kw):
    """Choice equal, weights within float32's roundings: exp 2 units, two
    divisions and the scale half a unit each, the sum's 36 terms at most
    half a unit each of a result below scale: 24 units of 2^-24 and the
    exponent's 2^-24 |z| (spread 8: another 16)."""
    zd = z.to(DEV)
    bd = None if bias is None else bias.to(DEV)
    gk = dict(kw)
    gk["group_best"] = gk.pop("best", 1)
    idx, w = M.router_select(zd, k, bias=bd, **gk)
    torch.cuda.synchronize()
    ri, rw = S.router_select(_f64(z), k, bias=None if bias is None else _f64(bias), **kw)
    np.testing.assert_array_equal(idx.cpu().numpy(), ri)
    tol = 64 * 2.0 ** -24
    np.testing.assert_allclose(_f64(w), rw, rtol=tol, atol=1e-38)
    return idx, w


CASES = [(1, 1, 1), (3, 2, 2), (7, 8, 3), (33, 31, 5), (16, 60, 4), (19, 64, 6), (21, 100, 8), (40, 256, 8),
         (9, 257, 32), (6, 512, 10), (5, 1000, 17), (4, 1024, 32)]


@pytest.mark.parametrize("T,E,k", CASES)
@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("score,biased,renorm", list(itertools.product(["softmax", "sigmoid"], [False, True], [False, True])))
def test_select(T, E, k, dt, score, biased, renorm):
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(7)) if biased else None
    _check(_logits(T, E, dt, T * E + k), k, bias, score=score, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("E,groups,top,k", [(8, 2, 1, 3), (64, 8, 4, 6), (256, 8, 4, 8), (60, 6, 2, 5), (96, 3, 2, 8),
                                            (1024, 32, 5, 16), (30, 30, 7, 7), (512, 4, 3, 8), (33, 11, 4, 9)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score,biased", list(itertools.product(["softmax", "sigmoid"], [False, True])))
def test_groups(E, groups, top, k, best, score, biased):
    if best > E // groups:
        pytest.skip("a group of one expert")
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(8)) if biased else None
    _check(_logits(37, E, F32, E + k), k, bias, score=score, groups=groups, top_groups=top, best=best)
    _check(_logits(21, E, BF, E + k), k, bias, score=score, groups=groups, top_groups=top, best=best)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_values_next_to_each_other(score):
    """Biases that bring scores within float32's error of each other: the
    choice is still that of the real numbers."""
    T, E = 512, 64
    g = torch.Generator().manual_seed(5)
    z = torch.randn((1, E), generator=g).expand(T, E).contiguous()
    s = torch.sigmoid(z.double()) if score == "sigmoid" else torch.softmax(z.double(), 1)
    bias = (0.75 - s[0]).float()             # every c within 2^-25 of 0.75
    _check(z, 8, bias, score=score)
    _check(z, 8, bias, score=score, groups=8, top_groups=3, best=2)
    z = z + 1e-6 * torch.randn((T, E), generator=g)
    _check(z, 8, bias, score=score)


def test_ties_go_to_the_lower_index():
    for E in (5, 64, 200, 256):
        z = torch.zeros(9, E)
        for kw in (dict(), dict(score="sigmoid")):
            idx, _ = _check(z, min(E, 8), **kw)
            assert idx.cpu().tolist() == [list(range(min(E, 8)))] * 9
            _check(z, min(E, 8), torch.zeros(E), **kw)
        z[:, 1::2] = -0.0
        _check(z, min(E, 8))
    z = torch.zeros(4, 64)
    _check(z, 8, groups=8, top_groups=2, best=2)
    _check(z, 8, torch.zeros(64), groups=8, top_groups=2, best=2, score="sigmoid")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_masks_infinities_and_nan(score, biased, renorm):
    E, k = 48, 4
    z = _logits(12, E, F32, 4)
    z[0] = -np.inf                                        # nothing left
    z[1] = torch.finfo(F32).min
    z[2] = torch.finfo(BF).min
    z[3, 3:] = -np.inf                                    # fewer than k
    z[4, 1:] = torch.finfo(F32).min
    z[5, ::2] = np.nan
    z[6] = np.nan
    z[7, 5], z[7, 9] = np.inf, np.inf
    z[8] = z[8] * 1e4
    z[9] = -1e3                                           # sigmoid underflows
    z[10, :] = 88.0
    z[11, 7] = 1e38
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(7)) if biased else None
    if biased:
        bias[11], bias[12] = -np.inf, np.nan
    _check(z, k, bias, score=score, renorm=renorm)
    _check(z, k, bias, score=score, renorm=renorm, groups=6, top_groups=2, best=2)
    _check(z, k, bias, score=score, renorm=renorm, groups=4, top_groups=2, best=1)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 3, 2), (33, 60, 4), (17, 64, 8), (40, 256, 8), (3, 1001, 32), (6, 1024, 10)])
@pytest.mark.parametrize("dt,ot", [(F32, F32), (F32, BF), (BF, BF), (BF, F32)])
@pytest.mark.parametrize("score,renorm", list(itertools.product(["softmax", "sigmoid"], [False, True])))
def test_gradient(T, E, k, dt, ot, score, renorm):
    z = _logits(T, E, dt, T + E)
    dw = torch.randn((T, k), generator=torch.Generator().manual_seed(2))
    idx, w = M.router_select(z.to(DEV), k, score=score, renorm=renorm, scale=2.5)
    got = M.router_select_bwd(z.to(DEV), idx, w, dw.to(DEV), score=score, renorm=renorm, scale=2.5, dtype=ot)
    ref = S.router_select_bwd(_f64(z), idx.cpu().numpy(), _f64(dw), score, renorm, 2.5)
    # terms of at most w max|dw| 2 each, with 64 units for the weight as above,
    # the dot's k roundings and the share's exp and sum: 256 units of that scale;
    # a bf16 output half a step of its value
    scale = 2 * 2.5 * np.abs(_f64(dw)).max(1, keepdims=True) + 0 * ref
    tol = 256 * 2.0 ** -24 * scale + (2.0 ** -8 * np.abs(ref) if ot is BF else 0)
    assert (np.abs(_f64(got) - ref) <= tol).all()
    # added to what is there
    start = torch.randn((T, E), generator=torch.Generator().manual_seed(3)).to(ot)
    acc = start.to(DEV)
    assert M.router_select_bwd(z.to(DEV), idx, w, dw.to(DEV), score=score, renorm=renorm, scale=2.5, dlogits=acc,
                               accumulate=True) is acc
    ref = ref + _f64(start)
    tol = 256 * 2.0 ** -24 * scale + 2.0 ** -23 * np.abs(ref) + (2.0 ** -8 * np.abs(ref) if ot is BF else 0)
    assert (np.abs(_f64(acc) - ref) <= tol).all()


def test_gradient_of_ids_out_of_range_and_twice():
    z = _logits(3, 40, F32, 1).to(DEV)
    idx = torch.tensor([[3, -1, 3, 40], [-1, -1, -1, -1], [5, 7, 5, 5]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[0.25, 9, 0.5, 9], [9] * 4, [0.1, 0.2, 0.3, 0.4]], device=DEV)
    dw = torch.tensor([[1.0, np.nan, 2.0, np.nan], [1.0] * 4, [1.0, 2.0, 3.0, 4.0]], device=DEV)
    g = M.router_select_bwd(z, idx, w, dw, renorm=True)
    ref = torch.zeros(3, 40, dtype=torch.float64)
    dot = 0.25 * 1 + 0.5 * 2
    ref[0, 3] = 0.25 * (1 - dot) + 0.5 * (2 - dot)
    dot = 0.1 + 0.4 + 0.9 + 1.6
    ref[2, 5] = 0.1 * (1 - dot) + 0.3 * (3 - dot) + 0.4 * (4 - dot)
    ref[2, 7] = 0.2 * (2 - dot)
    # a handful of roundings of terms of at most 2
    assert float((g.double().cpu() - ref).abs().max()) <= 16 * 2.0 ** -24 * 4


def test_masked_logits_get_no_gradient():
    z = _logits(4, 20, F32, 1)
    z[0, 5:] = -np.inf
    z[1, 3] = np.nan
    z[2] = torch.finfo(F32).min
    for score, renorm in itertools.product(["softmax", "sigmoid"], [False, True]):
        idx, w = M.router_select(z.to(DEV), 8, score=score, renorm=renorm)
        g = M.router_select_bwd(z.to(DEV), idx, w, torch.ones_like(w), score=score, renorm=renorm).cpu()
        assert torch.isfinite(g).all()
        assert (g[0, 5:] == 0).all() and g[1, 3] == 0 and (g[2] == 0).all()


def test_rows_of_a_batch_taken_at_any_row():
    """A contiguous part of a batch begins at any row, so at any multiple of the type."""
    for E in (33, 60, 64):
        for dt in (F32, BF):
            z = _logits(20, E, dt, E).to(DEV)
            idx, w = M.router_select(z, 4)
            for r in (1, 2, 3):
                i2, w2 = M.router_select(z[r:], 4)
                assert torch.equal(i2, idx[r:]) and torch.equal(w2, w[r:])
                g = M.router_select_bwd(z, idx, w, w * w, renorm=False, dtype=dt)
                out = torch.zeros_like(z)
                M.router_select_bwd(z[r:], idx[r:], w[r:], (w * w)[r:], renorm=False, dlogits=out[r:])
                assert torch.equal(out[r:], g[r:]) and (out[:r] == 0).all()


def test_no_tokens_and_reruns():
    z = torch.empty(0, 8, device=DEV)
    idx, w = M.router_select(z, 2)
    assert idx.shape == (0, 2) and M.router_select_bwd(z, idx, w, w).shape == (0, 8)
    z = _logits(3000, 256, F32, 3).to(DEV)
    b = (0.05 * torch.randn(256)).to(DEV)
    one = M.router_select(z, 8, score="sigmoid", bias=b, groups=8, top_groups=4, group_best=2)
    for _ in range(3):
        two = M.router_select(z, 8, score="sigmoid", bias=b, groups=8, top_groups=4, group_best=2)
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


def test_the_same_choice_as_the_plain_router():
    z = _logits(300, 256, F32, 9).to(DEV)
    i1, p1 = M.router_topk(z, 8)
    i2, p2 = M.router_select(z, 8)
    assert torch.equal(i1, i2)
    # both: exp 2 units, a sum of 8 and a division
    assert float((p1 - p2).abs().max()) <= 32 * 2.0 ** -24
