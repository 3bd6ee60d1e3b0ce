"""Tensors of more than 2^31 elements through the operators around the expert
MLP: rows before and after the 32-bit boundary against plain float64 values
of those rows.  (Tolerances: those of test_gpu_loss.py and test_gpu_linear.py,
for the sampled rows.)"""
import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu


def _rows(n, width):
    """Rows around element 2^31 of a [n, width] tensor, and its ends."""
    b = (1 << 31) // width
    assert b + 2 < n
    return [0, b - 1, b, b + 1, n - 1]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def test_router_losses():
    import dropless_grouped_gemm_gb300 as M
    T, E, k = (1 << 21) + 37, 1024, 2
    z = torch.randn((T, E), generator=_gen(1), device="cuda")
    idx = torch.randint(0, E, (T, k), generator=_gen(2), device="cuda", dtype=torch.int32)
    idx[:, 1] = (idx[:, 0] + 1) % E
    p = torch.full((T, k), 0.5, device="cuda")
    dp = torch.randn((T, k), generator=_gen(3), device="cuda") * 1e-6
    r = M.router_loss(z, idx)
    assert int(r["err"].item()) == 0 and int(r["n_valid"].item()) == T
    assert int(r["counts"].sum().item()) == T * k
    assert torch.equal(r["counts"][0], torch.bincount(idx.reshape(-1).long(), minlength=E).int())
    # float64 sums over the whole tensor, a block of tokens at a time
    sums, zsq = torch.zeros(E, device="cuda", dtype=torch.float64), 0.0
    for a in range(0, T, 1 << 17):
        lse = torch.logsumexp(z[a:a + (1 << 17)].double(), 1)
        sums += torch.exp(z[a:a + (1 << 17)].double() - lse[:, None]).sum(0)
        zsq += float(lse.square().sum())
    bal = float((r["counts"][0].double() * sums).sum()) * E / (k * T * T)
    # a lane adds up to 7,000 tokens in float32: an error that random signs keep
    # below sqrt(7000) u, and u per addition after it
    loss = r["loss"].tolist()
    assert abs(loss[0] - bal) <= 1e-5 * bal and abs(loss[1] - zsq / T) <= 1e-5 * zsq / T
    dl = torch.tensor([1.0, 1.0], device="cuda")
    g = M.router_loss_bwd(z, idx, r, dl, p, dp)
    w = r["counts"][0].double().cpu().numpy() * E / (k * float(T) * T)
    for t in _rows(T, E):
        zt = z[t].double().cpu().numpy()
        lse = np.log(np.exp(zt - zt.max()).sum()) + zt.max()
        assert abs(r["lse"][t].item() - lse) <= 48 * 2.0 ** -24 + 2 * 2.0 ** -24 * abs(lse)
        P = np.exp(zt - lse)
        d = P * (w - (P * w).sum() + 2 * lse / T)
        mag = P * (w + (P * w).sum() + 2 * abs(lse) / T)
        q = dp[t].double().cpu().numpy()
        for j in range(k):
            d[idx[t, j].item()] += 0.5 * (q[j] - 0.5 * q.sum())
            mag[idx[t, j].item()] += 0.5 * (abs(q[j]) + 0.5 * np.abs(q).sum())
        assert np.all(np.abs(g[t].cpu().numpy() - d) <= 96 * 2.0 ** -24 * mag), t


@pytest.mark.parametrize("f32", [False, True])
def test_linear_output(f32):
    import dropless_grouped_gemm_gb300 as M
    rows, K, N = 33000, 64, 65536 + 64
    a = torch.randn((rows, K), generator=_gen(4), device="cuda").bfloat16()
    B = (torch.randn((1, K, N), generator=_gen(5), device="cuda") * 0.1).bfloat16()
    b = torch.randn((1, N), generator=_gen(6), device="cuda").bfloat16()
    out, z, err = M.grouped_linear(a, None, B, "relu", b, save_z=not f32,
                                   out_dtype=torch.float32 if f32 else torch.bfloat16)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    at = _rows(rows, N)
    want = a[at].double() @ B[0].double() + b.double()
    mag = (K / 16 + 16) * 2.0 ** -22 * (a[at].abs().double() @ B[0].abs().double() + b.abs().double())
    step = 2.0 ** -24 if f32 else 2.0 ** -8
    got = out[at].double()
    assert bool(((got - want.clamp(min=0)).abs() <= mag + step * (want.abs() + mag)).all())
    if not f32:
        assert bool(((z[at].double() - want).abs() <= mag + step * (want.abs() + mag)).all())
        # the backward of the same rows: a million gradients a row
        dout = torch.randn((rows, N), generator=_gen(7), device="cuda").bfloat16()
        dz, da, dB, db, err = M.grouped_linear_bwd(dout, a, None, B, "relu", z, True)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        wz = torch.where(z[at] > 0, dout[at], torch.zeros_like(dout[at]))
        assert torch.equal(dz[at], wz)
        wa = wz.double() @ B[0].double().T
        amag = (N / 16 + 16) * 2.0 ** -22 * (wz.abs().double() @ B[0].abs().double().T)
        assert bool(((da[at].double() - wa).abs() <= amag + 2.0 ** -8 * wa.abs()).all())
        col = [0, 12345, N - 1]
        wb = torch.where(z[:, col] > 0, dout[:, col], torch.zeros_like(dout[:, col])).double()
        bmag = (24 + rows / 128 / 8 + 8) * 2.0 ** -24 * wb.abs().sum(0)
        assert bool(((db[0, col].double() - wb.sum(0)).abs() <= bmag).all())


def test_checkpoints():
    import dropless_grouped_gemm_gb300 as M
    T, d, k = 270_000, 8192, 1
    x = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    for a in range(0, T, 1 << 15):
        x[a:a + (1 << 15)] = torch.randn((min(1 << 15, T - a), d), generator=_gen(a), device="cuda")
    q, s = M.checkpoint_pack(x)
    v = M.checkpoint_unpack(q, s)
    por = torch.arange(T, dtype=torch.int32, device="cuda").flip(0).contiguous()
    y = M.permute_checkpoint(q, s, por, k, row_of_pair=por)      # a reversal is its own inverse
    torch.cuda.synchronize()
    at = _rows(T, d)
    oq, os_ = O.checkpoint_pack(x[at].double().cpu().numpy())
    assert np.array_equal(q[at].cpu().numpy(), oq) and np.array_equal(s[at].cpu().numpy(), os_)
    assert np.array_equal(v[at].double().cpu().numpy(), O.checkpoint_unpack(oq, os_))
    assert torch.equal(y[[T - 1 - t for t in at]], v[at])
