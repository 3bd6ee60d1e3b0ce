"""Scores next to each other at other widths than 64 experts and 8 picks: no
lane left for the first one behind 32 picks, keys that hide more bits, bf16
logits with a bias, neighbours that only swap (moe_router_select)."""
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


def _same(z, k, score, bias, groups=1, top=None, best=1):
    idx, w = M.router_select(z.to(DEV), k, score=score, bias=None if bias is None else bias.to(DEV), groups=groups, top_groups=top,
                             group_best=best)
    ri, rw = S.router_select(_f64(z), k, score, None if bias is None else _f64(bias), groups, top, best)
    np.testing.assert_array_equal(idx.cpu().numpy(), ri)
    # (exp 2 units, two divisions, a sum of up to 32 terms: 64 units of 2^-24 as
    # for any logits of this size)
    np.testing.assert_allclose(_f64(w), rw, rtol=64 * 2.0 ** -24, atol=1e-38)


WIDTHS = [(20, 1), (20, 19), (32, 31), (48, 32), (64, 32), (100, 9), (128, 32), (256, 8), (256, 32), (300, 32), (512, 8), (512, 32),
          (700, 5), (1024, 8), (1024, 31), (1024, 32)]


@pytest.mark.parametrize("E,k", WIDTHS)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dt", [F32, BF])
def test_biased_scores_within_a_few_units(E, k, score, dt):
    T = 48
    g = torch.Generator().manual_seed(E * k)
    z = torch.randn((1, E), generator=g).to(dt).expand(T, E).contiguous()
    s = torch.sigmoid(z.double()) if score == "sigmoid" else torch.softmax(z.double(), 1)
    bias = (0.75 - s[0]).float()                          # every c within 2^-25 of 0.75
    _same(z, k, score, bias)
    _same(z, k, score, bias + 2e-6 * torch.randn(E, generator=g))
    if dt is F32:
        _same(z + 1e-6 * torch.randn((T, E), generator=g), k, score, bias)
        # a few near ones around the last pick, the others apart
        far = bias + 0.1 * torch.randn(E, generator=g).abs().floor()
        _same(z + 1e-6 * torch.randn((T, E), generator=g), k, score, far)
    else:
        _same((z.float() * (1 + 2.0 ** -8 * torch.randint(-1, 2, (T, E), generator=g))).to(BF), k, score, bias)


@pytest.mark.parametrize("E,k", WIDTHS)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_logits_within_the_bits_that_keys_hide(E, k, score):
    """Without a bias the order is that of the logits: float32 neighbours."""
    T = 64
    g = torch.Generator().manual_seed(E + k)
    base = 1.0 + torch.rand((T, 1), generator=g)
    for step in (1, 3, 40):
        z = base + step * 2.0 ** -23 * torch.randint(-8, 9, (T, E), generator=g)
        _same(z, k, score, None)
        _same(-z, k, score, None)
    z = base + torch.rand((T, E), generator=g)
    z[:, ::2] = z[:, 1::2] if E % 2 == 0 else z[:, ::2]    # ties in pairs
    _same(z, k, score, None)
    z[:, ::2] += 2.0 ** -22
    _same(z, k, score, None)


@pytest.mark.parametrize("E,groups,top,k", [(256, 8, 4, 32), (512, 8, 4, 8), (512, 16, 2, 32), (1024, 8, 3, 8), (1024, 32, 16, 32), (300, 6, 3, 32),
                                            (640, 5, 2, 10)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
def test_groups_within_a_few_units(E, groups, top, k, score, best):
    T = 40
    g = torch.Generator().manual_seed(E + groups)
    z = torch.randn((1, E), generator=g)
    s = torch.sigmoid(z.double()) if score == "sigmoid" else torch.softmax(z.double(), 1)
    bias = (0.75 - s[0]).float()
    zn = z + 1e-6 * torch.randn((T, E), generator=g)
    _same(zn, k, score, bias, groups, top, best)
    _same(zn, k, score, None, groups, top, best)
    _same((z + 0.3 * torch.randn((T, E), generator=g)).to(BF), k, score, bias, groups, top, best)


def test_neighbours_that_only_swap():
    """The picks are clear, two of them within float32's error."""
    g = torch.Generator().manual_seed(9)
    for score in ("softmax", "sigmoid"):
        for E, k in ((64, 4), (256, 8), (1024, 32)):
            z = torch.randn((200, E), generator=g)
            s = torch.sigmoid(z.double()) if score == "sigmoid" else torch.softmax(z.double(), 1)
            bias = 0.05 * torch.randn(E, generator=g).double()
            # experts 2i and 2i + 1 get the same c, to a unit, in the first row; near it in its copies
            bias[1::2] = s[0, 0::2] + bias[0::2] - s[0, 1::2]
            z = z[:1] + 3e-7 * torch.randn((200, E), generator=g)
            _same(z, k, score, bias.float())
