"""Rows of equal logits (a gate that starts at zero, padding) with groups: the
choice, and that it takes no second look at the rows (moe_router_select)."""
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


@pytest.mark.parametrize("E,groups,top,k", [(64, 8, 4, 6), (256, 8, 4, 8), (60, 6, 2, 5), (96, 3, 2, 8), (1024, 32, 5, 32), (30, 30, 7, 7)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dt", [F32, BF])
def test_equal_groups(E, groups, top, k, score, dt):
    n = E // groups
    g = torch.Generator().manual_seed(E)
    base = torch.randn(n, generator=g)
    z = torch.zeros(24, E)
    z[1] = 3.25
    z[2] = base.repeat(groups)                            # each group the same
    z[3] = z[2]
    z[3, n:2 * n] += 1e-6                                 # one a little above
    z[4] = z[2]
    z[4, -n:] += 1e-6
    z[5, 0], z[5, E - 1] = 1e-7, 2e-7
    z[6] = z[2]
    z[6, :n] = z[6, :n].flip(0)                           # equal sums, other places
    z[7] = -float("inf")
    z[8, ::2] = -float("inf")
    z[9, n:] = float("nan")
    z[10, 1::2] = -0.0
    z[11:] = z[2]
    z[11:] += 1e-7 * torch.randn((13, E), generator=g)
    z = z.to(dt)
    same, other = torch.zeros(E), 0.1 * torch.randn(n, generator=g).repeat(groups)
    masked = other.clone()
    masked[::n] = -float("inf")
    near = other + 1e-7 * torch.randn(E, generator=g)
    for bias in (None, same, other, masked, near):
        for best in (1, 2)[:n]:
            idx, _ = M.router_select(z.to(DEV), k, score=score, bias=None if bias is None else bias.to(DEV), groups=groups, top_groups=top,
                                     group_best=best)
            ri, _ = S.router_select(_f64(z), k, score, None if bias is None else _f64(bias), groups, top, best)
            np.testing.assert_array_equal(idx.cpu().numpy(), ri)


def _time(f):
    f()
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    best = float("inf")
    for _ in range(10):
        a.record()
        for _ in range(4):
            f()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("best", [1, 2])
def test_rows_of_zeros_take_no_second_look(biased, best):
    """In 64 bits 65,536 rows of 256 take some thirty times as long as usual, by
    the short way below twice; five times tells the two apart."""
    z = torch.randn((65536, 256), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    bias = torch.zeros(256, device=DEV) if biased else None
    out = M.router_select(z, 8, score="sigmoid", bias=bias, groups=8, top_groups=4, group_best=best)
    call = lambda x: M.router_select(x, 8, score="sigmoid", bias=bias, groups=8, top_groups=4, group_best=best, topk_idx=out[0], probs=out[1])  # noqa: E731
    usual = _time(lambda: call(z))
    zero = torch.zeros_like(z)
    assert _time(lambda: call(zero)) < 5 * usual
