"""The tensor scale of a ragged buffer: of the experts' rows, whatever lies
in the others (moe_fp4_tensor_scale_rows)."""
import numpy as np
import pytest
import torch

import dropless_grouped_gemm_gb300 as M
from oracle import fp4 as O

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
DEV = "cuda"


def _rows(rows, K, seed, std=1.0):
    return (std * torch.randn((rows, K), generator=torch.Generator().manual_seed(seed))).to(BF)


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("offsets,K", [([0, 7], 64), ([0, 5, 5, 133, 300], 192), ([0, 0, 0], 128), ([0, 1, 2, 3], 7168), ([0, 5000, 20000], 320)])
@pytest.mark.parametrize("other", [1e30, float("inf"), float("nan"), 0.0])
def test_the_experts_rows_alone(offsets, K, other):
    last = offsets[-1]
    x = _rows(last + 50, K, last, 0.01)
    x[last:] = other
    err = torch.zeros(1, dtype=I32, device=DEV)
    off = torch.tensor(offsets, dtype=I32, device=DEV)
    t = M.fp4_tensor_scale(x.to(DEV), offsets=off, err=err)
    assert t.shape == (1,) and float(t) == O.tensor_scale(_f64(x[:last])) and int(err) == 0
    if last:
        x[last // 2, K - 1], x[0, 0] = float("nan"), -float("inf")       # (not finite: left out)
        assert float(M.fp4_tensor_scale(x.to(DEV), offsets=off)) == O.tensor_scale(_f64(x[:last]))


def test_many_experts():
    n = torch.randint(0, 40, (1024,), generator=torch.Generator().manual_seed(1))
    off = torch.zeros(1025, dtype=I32)
    off[1:] = torch.cumsum(n, 0)
    x = _rows(int(off[-1]) + 9, 64, 2)
    x[int(off[-1]) - 1, 63] = 300
    x[int(off[-1]):] = 1e30
    assert float(M.fp4_tensor_scale(x.to(DEV), offsets=off.to(DEV))) == O.tensor_scale([300.0])


def test_offsets_that_are_not_in_order():
    x = _rows(300, 128, 1)
    x[:3] = 1e3
    x[250:] = 1e6
    for off in ([0, 200, 100, 250], [0, -5, 100, 200], [3, 100, 200, 250], [0, 100, 200, 400], [7, 2, 1, 250], [0, 240, 100, 50]):
        safe = np.maximum.accumulate(np.clip(off, 0, 300))
        err = torch.zeros(1, dtype=I32, device=DEV)
        t = M.fp4_tensor_scale(x.to(DEV), offsets=torch.tensor(off, dtype=I32, device=DEV), err=err)
        assert int(err) == M.DEV_BAD_OFFSETS and float(t) == O.tensor_scale(_f64(x)[safe[0]:safe[-1]]), off


def test_no_rows_a_given_scale_and_a_graph():
    off = torch.zeros(3, dtype=I32, device=DEV)
    assert float(M.fp4_tensor_scale(torch.empty(0, 64, dtype=BF, device=DEV), offsets=off)) == 1
    x = torch.full((40, 64), 7.0, dtype=BF, device=DEV)
    t = torch.full((1,), -3.0, device=DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)
    assert M.fp4_tensor_scale(x, offsets=off, t=t, err=err) is t and float(t) == 1
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            M.fp4_tensor_scale(x, offsets=off, t=t, err=err)
    for n, v in ((10, 100.0), (40, 1.0), (0, 5.0), (39, 2688.0)):
        off.copy_(torch.tensor([0, n // 2, n], dtype=I32))
        x[:n], x[n:] = v, 1e30
        g.replay()
        torch.cuda.synchronize()
        assert float(t) == (O.tensor_scale([v]) if n else 1) and int(err) == 0


def test_the_scale_of_a_products_own_output():
    """A buffer longer than the experts' rows, from one product to the next in
    4 bits: what the rows behind held does not reach the result."""
    g = torch.Generator(device=DEV).manual_seed(3)
    offsets, K, N = [0, 30, 30, 101], 256, 320
    off = torch.tensor(offsets, dtype=I32, device=DEV)
    rows = offsets[-1] + 60
    x = torch.randn((rows, K), generator=g, device=DEV).to(BF)
    w = M.fp4_quantize_weights((0.1 * torch.randn((3, N, K), generator=g, device=DEV)).to(BF), along="cols")
    w2 = M.fp4_quantize_weights((0.1 * torch.randn((3, K, N), generator=g, device=DEV)).to(BF), along="cols")
    outs = []
    for behind in (0.0, 1e30):
        y = torch.full((rows, N), behind, dtype=BF, device=DEV)
        M.fp4_linear(M.fp4_quantize(x, off), off, w, act="silu", out=y)
        t = M.fp4_tensor_scale(y, offsets=off)
        out, _, err = M.fp4_linear(M.fp4_quantize(y, off, scale=t), off, w2, a_scale=t)
        assert int(err) == 0
        outs.append((float(t), out[:offsets[-1]]))
    assert outs[0][0] == outs[1][0] and torch.equal(outs[0][1], outs[1][1])
