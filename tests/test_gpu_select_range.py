"""Renormalised sigmoid weights of logits far below 0, where a float32 sigmoid
loses its bits (below -87) and then all of itself (below -88.7), and the
gradient that is built from them (moe_router_select, moe_router_select_bwd)."""
import numpy as np
import pytest
import torch

import dropless_grouped_gemm_gb300 as M
from oracle import select as S

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16
DEV = "cuda"


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _weights(z, scale):
    """scale s_j / sum_i s_i from the logarithms of the sigmoids, in 64 bits."""
    ls = np.where(z <= 0, z - np.log1p(np.exp(np.minimum(z, 0))), -np.log1p(np.exp(-np.maximum(z, 0))))
    w = np.exp(ls - ls.max(-1, keepdims=True))
    return scale * w / w.sum(-1, keepdims=True)


def _rows(dt):
    g = torch.Generator().manual_seed(3)
    z = torch.empty(64, 24)
    for r in range(40):                                   # at any depth that a 64-bit sigmoid has
        low = -80 - 600 * torch.rand(1, generator=g)
        z[r] = low + (20 if r % 2 else 1) * (torch.rand(24, generator=g) - 1)
    z[40] = -100 - 0.1 * torch.arange(24)
    z[41] = -88 - torch.arange(24) % 2                    # on both sides of float32's end
    z[42] = -88.7 - 0.01 * torch.arange(24)
    z[43] = -87 + 0.02 * torch.arange(24)                 # where the sigmoid becomes subnormal
    z[44] = -60 - 29 * (torch.arange(24) % 2)
    z[45] = -5 - 12 * torch.arange(24)
    z[46] = 3 - 12 * torch.arange(24)
    z[47] = 1e-3 - 90 * (torch.arange(24) % 3)
    z[48] = -87
    z[49] = -700
    z[50] = 0
    z[51:] = torch.randn(13, 24, generator=g) * 40 - 90
    return z.clamp(min=-700).to(dt)


def _tolerance(zc, w):
    """A term: the exponent's difference rounds by 2^-24 of it, exp 4 units of
    2^-24, 1 + e^z and a division 6 more; the sum of up to 32 terms 5, a
    division and the scale 2; numerator and sum both: 2 (|z - max| + 10) + 7
    units.  Below 2^-120 what is left of float32's range."""
    far = (zc.max(-1, keepdims=True) - zc).max(-1, keepdims=True)
    return (32 + 2 * far) * 2.0 ** -24 * w + 2.0 ** -120


@pytest.mark.parametrize("k", [1, 2, 5, 8])
@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("biased,groups", [(False, 1), (True, 1), (True, 4)])
def test_weights_of_low_logits(k, dt, biased, groups):
    z = _rows(dt)
    bias = 0.2 * torch.randn(24, generator=torch.Generator().manual_seed(5)) if biased else None
    kw = dict(groups=groups, top_groups=(groups + 1) // 2)
    idx, w = M.router_select(z.to(DEV), k, score="sigmoid", bias=None if bias is None else bias.to(DEV), group_best=1, scale=2.5, **kw)
    ri, _ = S.router_select(_f64(z), k, "sigmoid", None if bias is None else _f64(bias), best=1, scale=2.5, **kw)
    np.testing.assert_array_equal(idx.cpu().numpy(), ri)
    zc = np.take_along_axis(_f64(z), ri.astype(np.int64), 1)
    ref = _weights(zc, 2.5)
    assert (np.abs(_f64(w) - ref) <= _tolerance(zc, ref)).all()


def test_a_sigmoid_below_64_bits_counts_as_nothing():
    """As it is documented: at -709.79 and below a score is 0, and a sum of 0
    gives weights of 0; beside a larger one it has none either."""
    z = torch.full((4, 6), -709.8)
    z[1] = -3e4
    z[2, 2] = -709.7
    z[3, 1] = -709.0
    idx, w = M.router_select(z.to(DEV), 2, score="sigmoid")
    assert idx.cpu().tolist() == [[0, 1], [0, 1], [2, 0], [1, 0]]
    assert w.cpu().tolist() == [[0, 0], [0, 0], [1, 0], [1, 0]]


@pytest.mark.parametrize("dt", [F32, BF])
def test_gradient_of_low_logits(dt):
    k, scale = 4, 2.5
    z = _rows(dt)
    dw = torch.randn((z.shape[0], k), generator=torch.Generator().manual_seed(2))
    idx, w = M.router_select(z.to(DEV), k, score="sigmoid", scale=scale)
    got = _f64(M.router_select_bwd(z.to(DEV), idx, w, dw.to(DEV), score="sigmoid", scale=scale))
    i = idx.cpu().numpy().astype(np.int64)
    zc, d = np.take_along_axis(_f64(z), i, 1), _f64(dw)
    f = lambda x: (_weights(x, scale) * d).sum(1)  # noqa: E731
    ref = np.zeros_like(got)
    h = 1e-5
    for j in range(k):
        e = np.zeros_like(zc)
        e[:, j] = h
        ref[np.arange(len(zc)), i[:, j]] = (f(zc + e) - f(zc - e)) / (2 * h)
    rw = _weights(zc, scale)
    formula = rw * (d - (rw * d).sum(1, keepdims=True) / scale) / (1 + np.exp(np.minimum(zc, 700)))
    full = np.zeros_like(got)
    np.put_along_axis(full, i, formula, 1)
    # a term's weight as above, terms of at most 2 scale max|dw|; the differences'
    # own error h^2 of the third derivative and 2^-52 / h of f
    size = 2 * scale * np.abs(d).max(1, keepdims=True)
    far = (zc.max(1) - zc.min(1))[:, None]
    assert (np.abs(got - full) <= (256 + 4 * far) * 2.0 ** -24 * size).all()
    assert (np.abs(full - ref) <= 1e-8 * size).all()
