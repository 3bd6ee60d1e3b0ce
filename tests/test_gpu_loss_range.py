"""Router losses over the whole range of the logits: rows far from zero.

Tolerances, with u = 2^-24.  The exponents are 2^((v - m) log2 e): v - m is
exact for values within a factor of two of each other and otherwise rounded
once, so P is within 48u of itself plus 2u of |v - m| (below 64 where P is
above 2^-90), 176u in all, whatever the row's offset; the inputs are those
float32 values themselves.  lse = m + log sum: 2u of its magnitude and 48u."""
import numpy as np
import pytest
import torch

import oracle as O
from _helpers import cuda_i32

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
LARGE = [-5e9, -1e10, -3e10, -1e11, -1e12, -1e20, -1e30, -3e38, 1e10, 1e11, 1e30, 3e38]


def _rows(E, seed=3):
    """Rows of all-equal large logits, the same with one entry below the others,
    and ordinary ones between them."""
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((3 * len(LARGE), E)).astype(np.float32)
    for i, v in enumerate(LARGE):
        z[3 * i] = v
        z[3 * i + 1] = v
        z[3 * i + 1, i % E] = v - abs(v) * 2.0 ** -6
    return z


@pytest.mark.parametrize("E,dtype", [(8, torch.float32), (12, torch.float32), (60, torch.bfloat16),
                                     (64, torch.float32), (200, torch.float32), (256, torch.bfloat16),
                                     (520, torch.float32), (1023, torch.float32)])
def test_rows_of_large_logits(E, dtype):
    import dropless_grouped_gemm_gb300 as M
    k = 2
    zt = torch.from_numpy(_rows(E)).to(dtype)
    z = zt.double().numpy()
    assert np.isfinite(z).all()
    T = z.shape[0]
    idx = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    ref = O.router_loss(z, idx)
    assert ref["n_valid"].tolist() == [T]
    r = M.router_loss(zt.cuda(), cuda_i32(idx))
    torch.cuda.synchronize()
    lse = r["lse"].cpu().numpy().astype(np.float64)
    assert np.all(np.abs(lse - ref["lse"]) <= 48 * U + 2 * U * np.abs(ref["lse"]))
    assert r["n_valid"].cpu().tolist() == [T]
    assert r["counts"].cpu().tolist() == ref["counts"].tolist()
    got = r["loss"].cpu().numpy().astype(np.float64)
    assert abs(got[0] - ref["loss"][0]) <= 512 * U * ref["loss"][0]
    assert np.isposinf(got[1])                      # the mean of lse^2 is past float32


@pytest.mark.parametrize("v", [-1e9, -3e10, 1e11])
def test_both_losses_with_rows_padded_by_a_large_value(v):
    import dropless_grouped_gemm_gb300 as M
    T, E, k = 90, 48, 2
    z = np.random.default_rng(1).standard_normal((T, E)).astype(np.float32)
    z[60:] = v
    idx = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    ref = O.router_loss(z, idx)
    r = M.router_loss(torch.from_numpy(z).cuda(), cuda_i32(idx))
    torch.cuda.synchronize()
    assert r["counts"].cpu().tolist() == ref["counts"].tolist()
    got = r["loss"].cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - ref["loss"]) <= 512 * U * ref["loss"])
