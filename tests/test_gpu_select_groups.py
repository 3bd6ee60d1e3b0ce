"""The choice of groups by the sum of two scores of opposite signs: the sum is
small, the roundings are those of its terms (moe_router_select)."""
import numpy as np
import pytest
import torch

import dropless_grouped_gemm_gb300 as M
from oracle import select as S

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,groups,top,k,size", [(3000, 64, 8, 4, 6, 16.0), (1500, 256, 8, 4, 8, 16.0), (500, 1024, 8, 3, 8, 16.0),
                                                   (600, 96, 3, 1, 4, 100.0), (400, 512, 16, 8, 5, 3.0), (500, 60, 6, 2, 5, 30.0)])
def test_groups_whose_two_best_cancel(score, T, E, groups, top, k, size):
    """One expert of each group has a bias of `size`, the others minus that."""
    g = torch.Generator().manual_seed(E + groups)
    n = E // groups
    z = torch.randn((T, E), generator=g)
    bias = 0.01 * torch.randn(E, generator=g) - size
    bias[torch.randint(0, n, (groups,), generator=g) + n * torch.arange(groups)] += 2 * size
    kw = dict(score=score, groups=groups, top_groups=top)
    idx, _ = M.router_select(z.to(DEV), k, bias=bias.to(DEV), group_best=2, **kw)
    ri, _ = S.router_select(_f64(z), k, bias=_f64(bias), best=2, **kw)
    np.testing.assert_array_equal(idx.cpu().numpy(), ri)


def test_groups_that_a_bias_closes_are_in_no_doubt():
    """Groups pushed far down or up by their biases leave the others' order as
    exact as before."""
    g = torch.Generator().manual_seed(1)
    z = torch.randn((2000, 64), generator=g)
    bias = 0.05 * torch.randn(64, generator=g)
    bias[8:16] -= 1e9
    bias[32:40] += 1e6
    for score in ("sigmoid", "softmax"):
        idx, _ = M.router_select(z.to(DEV), 6, score=score, bias=bias.to(DEV), groups=8, top_groups=4, group_best=2)
        ri, _ = S.router_select(_f64(z), 6, score, _f64(bias), 8, 4, 2)
        np.testing.assert_array_equal(idx.cpu().numpy(), ri)
