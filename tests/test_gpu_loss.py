"""Router losses and their gradient (moe_router_loss, moe_router_loss_bwd)
against the oracle.

Tolerances, with u = 2^-24: an expf is within 2 ulp and a row's sum of at
most 32 values per lane and 5 shuffle steps, so P is within 48u of itself,
and lse within 48u + u |lse|.  A column sum adds one more rounding per token
of a warp, unit and lane of the finish (below 64 in these cases), and the
last sums below 64: losses within 256u of the sum of their terms'
magnitudes.  A gradient is P (w - dot + ...) + sum p (dp - mean): within 96u
of the same expression with every term's magnitude, plus half a bf16 step
where it is stored in bf16."""
import numpy as np
import pytest
import torch

import oracle as O
from _helpers import cuda_i32

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _inputs(seed, T, E, k, S, mask, dtype):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((T, E)) * 2.0 - 0.6 * np.log(1.0 + np.arange(E))
    z = torch.from_numpy(z).to(dtype)
    zf = z.double().numpy()
    idx = np.argsort(-zf, axis=1, kind="stable")[:, :k].astype(np.int32)
    seg = None
    if S > 1:
        seg = np.concatenate([[0], np.sort(rng.integers(0, T + 1, S - 1)), [T]]).astype(np.int32)
    m = (rng.random(T) > 0.25).astype(np.uint8) if mask else None
    p = rng.random((T, k)).astype(np.float32)
    p /= p.sum(axis=1, keepdims=True)
    dp = rng.standard_normal((T, k)).astype(np.float32)
    return z, zf, idx, seg, m, p, dp


def _cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


CASES = [
    # T, E, k, S, mask, dtype
    (1, 1, 1, 1, False, torch.float32),
    (1, 5, 2, 1, False, torch.float32),
    (7, 8, 3, 3, True, torch.float32),
    (64, 64, 2, 1, False, torch.float32),
    (333, 60, 4, 5, True, torch.bfloat16),
    (500, 33, 33, 1, False, torch.float32),      # odd E, every expert chosen
    (700, 256, 8, 40, True, torch.float32),      # segments in two groups of 32, some empty
    (257, 520, 8, 1, True, torch.bfloat16),
    (129, 1024, 40, 2, False, torch.float32),    # k above a warp
    (91, 1023, 5, 64, False, torch.bfloat16),
    (2600, 31, 2, 1, False, torch.bfloat16),     # several rounds of a unit
]


@pytest.mark.parametrize("T,E,k,S,mask,dtype", CASES)
def test_losses_and_gradient(T, E, k, S, mask, dtype):
    import dropless_grouped_gemm_gb300 as M
    z, zf, idx, seg, m, p, dp = _inputs(T + E, T, E, k, S, mask, dtype)
    ref = O.router_loss(zf, idx, seg, m)
    zc, ic, sc, mc = z.cuda(), cuda_i32(idx), _cuda(seg), _cuda(m)
    r = M.router_loss(zc, ic, sc, mc)
    r2 = M.router_loss(zc, ic, sc, mc)
    torch.cuda.synchronize()
    assert int(r["err"].item()) == 0
    assert r["counts"].cpu().tolist() == ref["counts"].tolist()
    assert r["n_valid"].cpu().tolist() == ref["n_valid"].tolist()
    lse = r["lse"].cpu().numpy().astype(np.float64)
    assert np.all(np.abs(lse - ref["lse"]) <= 48 * U + 2 * U * np.abs(ref["lse"]))
    loss = r["loss"].cpu().numpy().astype(np.float64)
    # every term of both sums is positive; lse^2 carries lse's error twice
    tol = 256 * U * ref["loss"]
    tol[1] += 2 * 50 * U * np.mean(np.abs(ref["lse"])) * (T / max(1, ref["n_valid"].sum()))
    assert np.all(np.abs(loss - ref["loss"]) <= tol)
    for name in ("loss", "lse"):
        assert torch.equal(r[name], r2[name])        # bitwise rerun

    dl = np.array([0.5, 0.25], np.float32)
    N = max(1, int(ref["n_valid"].sum()))
    got = {dt: M.router_loss_bwd(zc, ic, r, _cuda(dl), _cuda(p), _cuda(dp), sc, mc, dtype=dt)
           for dt in (torch.float32, torch.bfloat16)}
    bare = M.router_loss_bwd(zc, ic, r, _cuda(dl), seg_offsets=sc, token_mask=mc)
    torch.cuda.synchronize()
    want = O.router_loss_bwd(zf, idx, dl, p, dp, seg, m)
    want_bare = O.router_loss_bwd(zf, idx, dl, None, None, seg, m)
    # magnitudes of the terms
    P = np.exp(zf - ref["lse"][:, None])
    _, owner = O.ops._segments(T, seg)
    w = dl[0] * E * ref["counts"][np.maximum(owner, 0)] / (k * N * np.maximum(1, ref["n_valid"][np.maximum(owner, 0)])[:, None])
    mag = P * (w + (P * w).sum(axis=1, keepdims=True) + 2 * dl[1] * np.abs(ref["lse"][:, None]) / N)
    rmag = np.abs(p) * (np.abs(dp) + np.abs(p * dp).sum(axis=1, keepdims=True))
    mag_r = mag.copy()
    np.add.at(mag_r, (np.arange(T)[:, None], idx), rmag)
    err = lambda t, ref_: np.abs(t.float().cpu().numpy().astype(np.float64) - ref_)  # noqa: E731
    assert np.all(err(got[torch.float32], want) <= 96 * U * mag_r + 1e-38)
    assert np.all(err(bare, want_bare) <= 96 * U * mag + 1e-38)
    assert np.all(err(got[torch.bfloat16], want) <= 96 * U * mag_r + 2.0 ** -8 * np.abs(want) + 1e-38)


def test_rows_without_a_finite_logit_and_special_values():
    import dropless_grouped_gemm_gb300 as M
    T, E, k = 40, 12, 2
    rng = np.random.default_rng(5)
    z = rng.standard_normal((T, E)).astype(np.float32)
    z[3] = -np.inf                                  # a row that a mask empties
    z[4, 1:] = -np.inf
    z[5, :6] = np.finfo(np.float32).min             # the type's lowest value as a mask
    z[6] = np.finfo(np.float32).min
    idx = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    mask = np.ones(T, np.uint8)
    mask[9] = 0
    zm = z.copy()
    zm[9] = np.nan                                  # NaN in a masked place stays there
    r = M.router_loss(_cuda(zm), cuda_i32(idx), token_mask=_cuda(mask))
    g = M.router_loss_bwd(_cuda(zm), cuda_i32(idx), r, _cuda(np.ones(2, np.float32)),
                          token_mask=_cuda(mask))
    torch.cuda.synchronize()
    ref = O.router_loss(z, idx, None, mask)
    assert int(r["n_valid"].item()) == T - 3          # rows 3 and 6 are empty, 9 is masked
    assert r["counts"].cpu().tolist() == ref["counts"].tolist()
    want = ref["loss"]
    got = r["loss"].cpu().numpy()
    assert np.all(np.abs(got - want) <= 256 * U * np.abs(want))
    gg = g.cpu().numpy()
    assert np.isfinite(gg).all() and np.all(gg[[3, 6, 9]] == 0)
    assert np.isneginf(r["lse"][3].item()) and np.isneginf(r["lse"][6].item())
    # the same masks in bf16, whose lowest value is another one, and that in float32
    zb = torch.from_numpy(z).bfloat16()
    zb[5, :6] = torch.finfo(torch.bfloat16).min
    zb[6] = torch.finfo(torch.bfloat16).min
    ref = O.router_loss(zb.double().numpy(), idx, None, mask)
    for zz in (zb, zb.float()):
        r = M.router_loss(zz.cuda(), cuda_i32(idx), token_mask=_cuda(mask))
        torch.cuda.synchronize()
        assert int(r["n_valid"].item()) == T - 3
        got = r["loss"].cpu().numpy()
        assert np.all(np.abs(got - ref["loss"]) <= 256 * U * np.abs(ref["loss"]))
    # NaN in a valid row reaches the losses, and only that row's gradient
    z[2, 3] = np.nan
    r = M.router_loss(_cuda(z), cuda_i32(idx))
    g = M.router_loss_bwd(_cuda(z), cuda_i32(idx), r, _cuda(np.ones(2, np.float32)))
    torch.cuda.synchronize()
    assert np.isnan(r["loss"].cpu().numpy()).all()
    gg = np.isnan(g.cpu().numpy()).any(axis=1)
    assert gg[2] and gg.sum() == 1


def test_unrouted_and_bad_ids_and_offsets():
    import dropless_grouped_gemm_gb300 as M
    T, E, k = 50, 6, 3
    _, zf, idx, _, _, p, dp = _inputs(9, T, E, k, 1, False, torch.float32)
    z = zf.astype(np.float32)
    idx[4] = -1
    idx[7, 1] = -1
    seg = np.array([0, 20, 44], np.int32)           # tokens 44.. lie in no sequence
    ref = O.router_loss(z, idx, seg)
    r = M.router_loss(_cuda(z), cuda_i32(idx), _cuda(seg))
    g = M.router_loss_bwd(_cuda(z), cuda_i32(idx), r, _cuda(np.ones(2, np.float32)), _cuda(p),
                          _cuda(dp), _cuda(seg))
    torch.cuda.synchronize()
    assert int(r["err"].item()) == 0
    assert r["counts"].cpu().tolist() == ref["counts"].tolist()
    want = O.router_loss_bwd(z, idx, [1.0, 1.0], p, dp, seg)
    assert np.abs(g.cpu().numpy() - want).max() <= 96 * U * 8   # every term is below 2, four of them
    # a bad id is skipped and reported; bad offsets are corrected and reported
    bad = idx.copy()
    bad[2, 0] = E
    r = M.router_loss(_cuda(z), cuda_i32(bad))
    torch.cuda.synchronize()
    assert int(r["err"].item()) == M.DEV_BAD_EXPERT
    for off in ([0, 60, 50], [3, 20, 50], [0, 30, 20], [-1, 5, 50]):
        r = M.router_loss(_cuda(z), cuda_i32(idx), _cuda(np.array(off, np.int32)))
        torch.cuda.synchronize()
        assert int(r["err"].item()) == M.DEV_BAD_OFFSETS, off


@pytest.mark.parametrize("E,k", [(6, 4), (100, 12), (300, 40)])
def test_an_expert_chosen_twice_gets_both_terms(E, k):
    import dropless_grouped_gemm_gb300 as M
    T = 37
    _, zf, idx, _, _, p, dp = _inputs(13, T, E, k, 1, False, torch.float32)
    idx[::3, 1] = idx[::3, 0]
    idx[::5, 2:4] = idx[::5, :1]
    z = zf.astype(np.float32)
    ref = O.router_loss(z, idx)
    r = M.router_loss(_cuda(z), cuda_i32(idx))
    g = M.router_loss_bwd(_cuda(z), cuda_i32(idx), r, _cuda(np.ones(2, np.float32)), _cuda(p), _cuda(dp))
    again = M.router_loss_bwd(_cuda(z), cuda_i32(idx), r, _cuda(np.ones(2, np.float32)), _cuda(p), _cuda(dp))
    torch.cuda.synchronize()
    assert r["counts"].cpu().tolist() == ref["counts"].tolist()
    assert torch.equal(g, again)
    want = O.router_loss_bwd(z, idx, [1.0, 1.0], p, dp)
    # every term is below 4 in magnitude here, up to five add up
    assert np.abs(g.cpu().numpy() - want).max() <= 96 * U * 20


def test_no_tokens():
    import dropless_grouped_gemm_gb300 as M
    z = torch.empty((0, 16), device="cuda")
    i = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    r = M.router_loss(z, i)
    g = M.router_loss_bwd(z, i, r, torch.ones(2, device="cuda"))
    torch.cuda.synchronize()
    assert r["loss"].tolist() == [0.0, 0.0] and r["counts"].sum().item() == 0
    assert r["n_valid"].tolist() == [0] and g.shape == (0, 16)


def test_captures_into_a_graph_on_another_stream():
    import dropless_grouped_gemm_gb300 as M
    z, zf, idx, seg, m, p, dp = _inputs(11, 300, 64, 4, 3, True, torch.float32)
    zc, ic, sc, mc = z.cuda(), cuda_i32(idx), _cuda(seg), _cuda(m)
    dl, pc, dc = torch.tensor([1.0, 0.5], device="cuda"), _cuda(p), _cuda(dp)
    want = M.router_loss(zc, ic, sc, mc)
    wg = M.router_loss_bwd(zc, ic, want, dl, pc, dc, sc, mc)
    torch.cuda.synchronize()
    out = {n: torch.zeros_like(t) for n, t in want.items()}
    ws = torch.empty(M.router_loss_workspace_size(300, 64, 3), dtype=torch.uint8, device="cuda")
    dz = torch.zeros_like(wg)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        M.router_loss(zc, ic, sc, mc, out=out, workspace=ws)
        M.router_loss_bwd(zc, ic, out, dl, pc, dc, sc, mc, dlogits=dz)
    ws.fill_(0xFF)                                   # the workspace need not be initialised
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for n in ("loss", "counts", "lse", "n_valid"):
        assert torch.equal(out[n], want[n]), n
    assert torch.equal(dz, wg)
