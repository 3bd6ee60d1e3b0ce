"""The gradient of a whole layer's input through the 4-bit products against a
float64 composition on the same routing and 4-bit values, and against the bf16
layer's."""
import numpy as np
import pytest
import torch

import dropless_grouped_gemm_gb300 as M
import oracle as O
from oracle import fp4 as F
from test_gpu_fp4_block import Layer, _close, _f64, _held

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_gradient_of_the_layers_input(fmt):
    T, d, n, E, k = 300, 256, 128, 16, 3
    L = Layer(T, d, n, E, k, fmt, 4)
    idx, probs = M.router_select(L.logits, k, **L.route)
    r = M.route_offsets(idx, E)
    off, por, rop = r["offsets"], r["pair_of_row"], r["row_of_pair"]
    xp = M.permute(L.x, por, k, row_of_pair=rop)
    a, z, err = M.fp4_linear(M.fp4_quantize(xp, off, fmt=fmt), off, L.w1, fmt=fmt, act="swiglu", w_scale=L.t1, save_z=True)
    dout = torch.randn((T, d), generator=torch.Generator().manual_seed(9)).to(BF).to(DEV)
    dy = M.permute(dout, por, k, scale=probs.reshape(-1), row_of_pair=rop)
    _, da, _, _, _ = M.fp4_linear_bwd(dy, a, off, L.w2b, fmt=fmt, w_scale=L.t2, err=err)
    dz, dxp, _, _, _ = M.fp4_linear_bwd(da, xp, off, L.w1b, fmt=fmt, act="swiglu", z=z, w_scale=L.t1, err=err)
    dx = _f64(M.unpermute(dxp, rop, T, k)[0])
    assert int(err) == 0
    # float64: the rows' gradient from dz's 4-bit values, then summed over a
    # token's rows.  Each row's value is a bf16 (2^-9 of its 2-norm), the sum
    # another rounding: 0.004 of the 2-norm at most, where terms do not cancel
    # more than three random ones do
    o = off.cpu().tolist()
    g1 = _f64(dz)
    g1h = _held(g1, fmt, F.tensor_scale(g1) if fmt == "nvfp4" else 1.0)
    w1b = _f64(M.fp4_dequantize(L.w1b, fmt=fmt, scale=L.t1, dtype=F32))
    ref_rows = np.zeros((o[-1], d))
    for e in range(E):
        ref_rows[o[e]:o[e + 1]] = g1h[o[e]:o[e + 1]] @ w1b[e].T
    ref = ref_rows[rop.cpu().numpy().reshape(T, k)].sum(1)
    _close(dx, ref, "dx", 0.005)
    # the bf16 layer: the same formulas on the unquantised operands in float64
    ri, rw = idx.cpu().numpy(), _f64(probs)
    lay = O.route_offsets(ri, E, 1)
    x64, W1, W2 = _f64(xp), _f64(L.W1), _f64(L.W2)
    dy64 = O.permute(_f64(dout), lay["pair_of_row"], k) * rw.reshape(-1)[lay["pair_of_row"]][:, None]
    rows = np.zeros((o[-1], d))
    for e in range(E):
        i, j = o[e], o[e + 1]
        zz = x64[i:j] @ W1[e]
        g, u = zz[:, 0::2], zz[:, 1::2]
        sg = 1 / (1 + np.exp(-g))
        dh = dy64[i:j] @ W2[e].T
        dzz = np.empty_like(zz)
        dzz[:, 0::2], dzz[:, 1::2] = dh * u * sg * (1 + g * (1 - sg)), dh * g * sg
        rows[i:j] = dzz @ W1[e].T
    full = rows[rop.cpu().numpy().reshape(T, k)].sum(1)
    # E2M1's relative steps are 1/6 to 1/3 wide, so a value is off by 0.05 to 0.14
    # of itself, some 0.1 of a tensor's 2-norm, and an operand's error goes through
    # its product as it is.  Six reach dx: x and W1 through z (whose derivative
    # enters as a factor: twice), dy and W2, dz and W1: 0.1 sqrt(2 * 4 + 2 + 2) =
    # 0.35; half as much again for the blocks' scales, which MX rounds down to a
    # power of two
    err = float(np.linalg.norm(dx - full) / np.linalg.norm(full))
    assert err <= 0.55, err
