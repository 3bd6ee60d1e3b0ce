"""The linear operator where its offsets have to be corrected, and its
activations' derivatives over bf16's whole range.  The forward's tolerance is
that of its other tests: (K / 16 + 16) 2^-22 of the terms' magnitudes and half
a bf16 step."""
import numpy as np
import pytest
import torch

import oracle as O
import workloads as W
from _helpers import cuda_i32, f64

pytestmark = pytest.mark.gpu


def _corrected(off, M):
    return np.maximum.accumulate(np.clip(off, 0, M)).astype(np.int32)


# (the third: more blocks of rows than non-decreasing offsets can give)
BAD = [(40, [0, 40, 20, 40]), (300, [0, 150, 0, 150, 0, 300]), (3000, [0, 1500, 0, 1500, 0, 3000]),
       (3000, [0, 3000, 10, 2000, 3000]), (40, [2, 3, 4, 40]), (3000, [5, 700, 400, 3100]),
       (700, [0, -3, 4, 700])]


@pytest.mark.parametrize("act", ["none", "silu", "swiglu"])
@pytest.mark.parametrize("M,off", BAD)
def test_backward_corrects_bad_offsets_as_one(M, off, act):
    """dz, the bias gradient and both products take the same corrected rows:
    the results of the corrected offsets, bit for bit."""
    import dropless_grouped_gemm_gb300 as M_
    E, K, N = len(off) - 1, 64, 128
    n_out = N // 2 if act == "swiglu" else N
    a = W.normal((M, K), (31, W.X, 0), 1.0, "cuda")
    B = W.normal((E, K, N), (31, W.W2, 1), 0.05, "cuda")
    z = None if act == "none" else W.normal((M, N), (31, W.X, 5), 1.5, "cuda")
    dout = W.normal((M, n_out), (31, W.DO, 0), 1.0, "cuda")
    fixed = _corrected(off, M)

    def run(o):
        bufs = {"da": torch.full((M, K), 9.0, dtype=torch.bfloat16, device="cuda")}
        if act != "none":        # a row that dz leaves out shows in the products
            bufs["dz"] = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        return M_.grouped_linear_bwd(dout, a, cuda_i32(o), B, act, z, True, **bufs)

    good, bad = run(fixed), run(off)
    torch.cuda.synchronize()
    assert int(bad[-1].item()) == M_.DEV_BAD_OFFSETS
    assert int(good[-1].item()) == (0 if fixed[0] == 0 else M_.DEV_BAD_OFFSETS)
    lo, hi = int(fixed[0]), int(fixed[-1])
    for x, y, name in zip(good[:4], bad[:4], ("dz", "da", "dB", "dbias")):
        if name in ("dz", "da"):
            x, y = x[lo:hi], y[lo:hi]
        assert torch.isfinite(y).all(), name
        assert torch.equal(x, y), name


@pytest.mark.parametrize("M,K,N,dtype", [(40, 64, 128, torch.bfloat16), (40, 64, 128, torch.float32),
                                         (3000, 1024, 4096, torch.bfloat16)])
def test_forward_corrects_bad_offsets_alike_in_both_kernels(M, K, N, dtype):
    import dropless_grouped_gemm_gb300 as M_
    for off in ([2, 3, 4, M], [5, M // 2, M // 4, M + 100], [0, M, M // 2, M]):
        E = len(off) - 1
        a = W.normal((M, K), (32, W.X, 0), 1.0, "cuda")
        B = W.normal((E, K, N), (32, W.W2, 1), 0.05, "cuda")
        b = W.normal((E, N), (32, W.W2, 2), 0.5, "cuda")
        fixed = _corrected(off, M)
        out = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
        _, _, err = M_.grouped_linear(a, cuda_i32(off), B, "none", b, out=out)
        torch.cuda.synchronize()
        assert int(err.item()) == M_.DEV_BAD_OFFSETS
        assert (out[:fixed[0]] == 7.0).all()            # before the first expert: not written
        ends = [(r, e) for e in range(E) if fixed[e + 1] > fixed[e]
                for r in (int(fixed[e]), int(fixed[e + 1]) - 1)]
        rows, own = [r for r, _ in ends], [e for _, e in ends]
        want = np.stack([f64(a[r]) @ f64(B[e]) + f64(b[e]) for r, e in zip(rows, own)])
        mag = np.stack([np.abs(f64(a[r])) @ np.abs(f64(B[e])) + np.abs(f64(b[e])) for r, e in zip(rows, own)])
        got = out[rows].double().cpu().numpy()
        assert np.all(np.abs(got - want) <= (K / 16 + 16) * 2.0 ** -22 * mag + 2.0 ** -8 * np.abs(want))


@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu", "geglu"])
def test_derivatives_at_large_pre_activations(act):
    """Where the sigmoid is 0 or 1 to the last bit, phi' is too (past 1.8e19,
    z^2 is past float32).  Half a bf16 step, and the derivative's 2^-18 at the
    last three values, doubled by dout."""
    import dropless_grouped_gemm_gb300 as M_
    vals = [1e2, 1e9, 1e13, 1e18, 1.7e19, 2e19, 1e20, 1e30, 3e38]
    g = torch.tensor(vals + [-v for v in vals] + [0.0, 1.0, -1.0], device="cuda").bfloat16()
    M = g.numel()
    z = torch.full((M, 64), 0.5, dtype=torch.bfloat16, device="cuda")
    gated = act in ("swiglu", "geglu")
    z[:, ::2] = g[:, None]
    if not gated:
        z[:, 1::2] = g[:, None]
    dout = torch.full((M, 32 if gated else 64), 2.0, dtype=torch.bfloat16, device="cuda")
    a = torch.ones((M, 64), dtype=torch.bfloat16, device="cuda")
    B = torch.zeros((64, 64), dtype=torch.bfloat16, device="cuda")
    dz, _, _, _, _ = M_.grouped_linear_bwd(dout, a, None, B, act, z)
    torch.cuda.synchronize()
    near = O.dphi(np.array([0.0, 1.0, -1.0]), "swiglu" if act in ("silu", "swiglu") else "geglu")
    d = 2.0 * (0.5 if gated else 1.0) * np.concatenate([np.ones(len(vals)), np.zeros(len(vals)), near])
    got = f64(dz)[:, 0]
    assert np.all(np.abs(got - d) <= 2.0 ** -8 * np.abs(d) + 2.0 ** -17), got
