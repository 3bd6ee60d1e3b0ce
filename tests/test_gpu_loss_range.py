"""Router losses and their gradient over the whole range of the logits: rows
far from zero, and sequence offsets that have to be corrected.

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


def _cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


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


@pytest.mark.parametrize("E,dtype", [(8, torch.float32), (60, torch.bfloat16), (64, torch.float32),
                                     (200, torch.float32), (520, torch.float32), (1023, torch.float32)])
def test_gradient_of_rows_of_large_logits(E, dtype):
    import dropless_grouped_gemm_gb300 as M
    k = 2
    zt = torch.from_numpy(_rows(E)).to(dtype)
    z = zt.double().numpy()
    T = z.shape[0]
    idx = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    ref = O.router_loss(z, idx)
    r = M.router_loss(zt.cuda(), cuda_i32(idx))
    for dl in ([1.0, 0.0], [0.5, 0.25]):
        dl = np.array(dl, np.float32)
        g = M.router_loss_bwd(zt.cuda(), cuda_i32(idx), r, _cuda(dl)).cpu().numpy().astype(np.float64)
        want = O.router_loss_bwd(z, idx, dl)
        P, lse = O.ops._softmax(z)
        w = dl[0] * E * ref["counts"][0] / (k * T * T)
        mag = P * (w + (P * w).sum(axis=1, keepdims=True) + 2 * dl[1] * np.abs(lse[:, None]) / T)
        assert np.all(np.abs(g - want) <= 256 * U * mag + 1e-38), dl


@pytest.mark.parametrize("off", [0.0, 1e3, -1e4, 3e5])
@pytest.mark.parametrize("E", [8, 60, 256, 1000])
def test_gradient_does_not_depend_on_a_common_offset(E, off):
    """Logits on a grid that the offset leaves exact: the same softmax."""
    import dropless_grouped_gemm_gb300 as M
    T, k = 70, 2
    rng = np.random.default_rng(E)
    z = (np.round(rng.standard_normal((T, E)) * 64) / 32 + off).astype(np.float32)
    idx = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    ref = O.router_loss(z, idx)
    r = M.router_loss(_cuda(z), cuda_i32(idx))
    dl = np.array([1.0, 0.0], np.float32)
    g = M.router_loss_bwd(_cuda(z), cuda_i32(idx), r, _cuda(dl)).cpu().numpy().astype(np.float64)
    P, _ = O.ops._softmax(z)
    w = E * ref["counts"][0] / (k * T * T)
    mag = P * (w + (P * w).sum(axis=1, keepdims=True))
    assert np.all(np.abs(g - O.router_loss_bwd(z, idx, dl)) <= 256 * U * mag + 1e-38)


@pytest.mark.parametrize("off", [[0, 30, 10, 50], [0, 60, 50, 50], [3, 20, 10, 40], [0, -4, 25, 50],
                                 [0, 45, 0, 45, 0, 45, 50], [7, 3, 90, 12]])
def test_gradient_takes_the_corrected_offsets(off):
    """The forward clamps the offsets to [0, T], begins at 0 and takes their
    running maximum; the gradient has to be that of the same sequences."""
    import dropless_grouped_gemm_gb300 as M
    T, E, k = 50, 24, 3
    rng = np.random.default_rng(8)
    z = rng.standard_normal((T, E)).astype(np.float32)
    idx = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    fixed = np.maximum.accumulate(np.clip([0] + off[1:], 0, T)).astype(np.int32)
    dl = _cuda(np.array([1.0, 0.5], np.float32))
    a = M.router_loss(_cuda(z), cuda_i32(idx), cuda_i32(fixed))
    b = M.router_loss(_cuda(z), cuda_i32(idx), cuda_i32(off))
    ga = M.router_loss_bwd(_cuda(z), cuda_i32(idx), a, dl, seg_offsets=cuda_i32(fixed))
    gb = M.router_loss_bwd(_cuda(z), cuda_i32(idx), b, dl, seg_offsets=cuda_i32(off))
    torch.cuda.synchronize()
    assert int(a["err"].item()) == 0 and int(b["err"].item()) == M.DEV_BAD_OFFSETS
    for n in ("loss", "counts", "n_valid", "lse"):
        assert torch.equal(a[n], b[n]), n
    assert torch.equal(ga, gb)


@pytest.mark.parametrize("E,dtype", [(8, torch.float32), (60, torch.bfloat16), (200, torch.float32)])
def test_a_row_s_gradient_does_not_depend_on_its_neighbours(E, dtype):
    """Ordinary rows beside large, empty and NaN ones: the same bits."""
    import dropless_grouped_gemm_gb300 as M
    T, k = 64, 2
    rng = np.random.default_rng(E)
    z = torch.from_numpy(rng.standard_normal((T, E)) * 3.0).to(dtype).cuda()
    idx = z.float().topk(k).indices.int()
    mask = torch.ones(T, dtype=torch.uint8, device="cuda")
    odd = torch.arange(1, T, 2, device="cuda")
    mask[odd] = 0
    other = z.clone()
    other[odd] = torch.tensor([-1e30, float("-inf"), float("nan"), 1e9], device="cuda").to(dtype).repeat(8)[:, None]
    dl = _cuda(np.array([1.0, 0.5], np.float32))
    g = []
    for x in (z, other):
        r = M.router_loss(x, idx, token_mask=mask)
        g.append(M.router_loss_bwd(x, idx, r, dl, token_mask=mask))
    torch.cuda.synchronize()
    assert torch.equal(g[0], g[1])
