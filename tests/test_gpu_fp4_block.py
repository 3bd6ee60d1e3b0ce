"""The router's choice and the experts' products in 4 bits run together, as an
MoE layer uses them: choice by scores, routing layout, permute into 4 bits, two
products with the hidden activations in 4 bits, combine; and a training step.
Against a float64 composition on the same routing."""
import numpy as np
import pytest
import torch

import dropless_grouped_gemm_gb300 as M
import oracle as O
from oracle import fp4 as F
from oracle import select as S

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
DEV = "cuda"


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _held(x, fmt, t=1.0):
    return F.values(*F.quantize(x, fmt, t), fmt, t)


def _close(got, ref, name, share):
    """Within `share` of the result's 2-norm: half a bf16 step of each value and
    what the intermediate roundings that land on the other side of a border move
    (a code's step is up to 1/2 of a value, and float32 accumulation moves 1 in
    10^4 of them across: 0.5 sqrt(1e-4) = 0.005 at most)."""
    err = float(np.linalg.norm(got - ref) / np.linalg.norm(ref))
    assert err <= share, (name, err)


class Layer:
    def __init__(self, T, d, n, E, k, fmt, seed=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.T, self.d, self.n, self.E, self.k, self.fmt = T, d, n, E, k, fmt
        self.x = r(T, d).to(BF).to(DEV)
        self.logits = (r(T, E) - 0.3 * torch.arange(E)[None] / E).to(DEV)
        self.bias = (0.05 * r(E)).to(DEV)
        self.W1 = (r(E, d, 2 * n) * d ** -0.5).to(BF).to(DEV)
        self.W2 = (r(E, n, d) * n ** -0.5).to(BF).to(DEV)
        self.t1, self.t2, self.t1b, self.t2b = ((M.fp4_tensor_scale(w, per_expert=True) if fmt == "nvfp4" else None)
                                                for w in (self.W1, self.W2, self.W1, self.W2))
        self.w1 = M.fp4_quantize_weights(self.W1, fmt=fmt, along="rows", scale=self.t1)
        self.w2 = M.fp4_quantize_weights(self.W2, fmt=fmt, along="rows", scale=self.t2)
        self.w1b = M.fp4_quantize_weights(self.W1, fmt=fmt, along="cols", scale=self.t1)
        self.w2b = M.fp4_quantize_weights(self.W2, fmt=fmt, along="cols", scale=self.t2)
        self.route = dict(score="sigmoid", bias=self.bias, groups=4, top_groups=2, group_best=2, scale=2.5)

    def forward(self, x, logits):
        """Serving: the hidden activations stay in 4 bits."""
        idx, probs = M.router_select(logits, self.k, **self.route)
        r = M.route_offsets(idx, self.E)
        x4 = M.fp4_permute(x, r["pair_of_row"], self.k, r["offsets"], fmt=self.fmt, row_of_pair=r["row_of_pair"])
        h4, _, err = M.fp4_linear(x4, r["offsets"], self.w1, fmt=self.fmt, act="swiglu", w_scale=self.t1, out_dtype="fp4")
        y, _, _ = M.fp4_linear(h4, r["offsets"], self.w2, fmt=self.fmt, w_scale=self.t2, err=err)
        out, _ = M.unpermute(y, r["row_of_pair"], self.T, self.k, probs=probs)
        return out, idx, probs, r, err


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,d,n,E,k", [(1, 128, 64, 16, 2), (37, 256, 192, 32, 4), (900, 512, 256, 8, 2)])
def test_forward(fmt, T, d, n, E, k):
    L = Layer(T, d, n, E, k, fmt)
    out, idx, probs, r, err = L.forward(L.x, L.logits)
    torch.cuda.synchronize()
    assert int(err) == 0
    ri, rw = S.router_select(_f64(L.logits), k, "sigmoid", _f64(L.bias), 4, 2, 2, scale=2.5)
    np.testing.assert_array_equal(idx.cpu().numpy(), ri)
    lay = O.route_offsets(ri, E, 1)
    off = lay["offsets"]
    xp = _held(O.permute(_f64(L.x), lay["pair_of_row"], k), fmt)
    w1 = _f64(M.fp4_dequantize(L.w1, fmt=fmt, scale=L.t1, dtype=F32))
    w2 = _f64(M.fp4_dequantize(L.w2, fmt=fmt, scale=L.t2, dtype=F32))
    y = np.zeros((off[-1], d))
    for e in range(E):
        a, b = off[e], off[e + 1]
        if b > a:
            z = xp[a:b] @ w1[e].T
            h = z[:, 0::2] / (1 + np.exp(-z[:, 0::2])) * z[:, 1::2]
            y[a:b] = _held(h, fmt) @ w2[e].T
    ref = O.unpermute(y, lay["row_of_pair"], T, k, rw)
    _close(_f64(out), ref, "out", 0.01)


def test_in_a_graph_with_other_tokens():
    L = Layer(200, 256, 128, 32, 4, "nvfp4")
    x, logits = L.x.clone(), L.logits.clone()
    L.forward(x, logits)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out, _, _, _, err = L.forward(x, logits)
    torch.cuda.synchronize()
    for seed in (1, 2):
        other = Layer(200, 256, 128, 32, 4, "nvfp4", seed)
        x.copy_(other.x)
        logits.copy_(other.logits)
        g.replay()
        torch.cuda.synchronize()
        assert int(err) == 0 and torch.equal(out, L.forward(x, logits)[0])


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_training_step(fmt):
    T, d, n, E, k = 300, 256, 128, 16, 3
    L = Layer(T, d, n, E, k, fmt, 4)
    idx, probs = M.router_select(L.logits, k, **L.route)
    loss = M.router_loss(L.logits, idx)
    r = M.route_offsets(idx, E)
    off, por, rop = r["offsets"], r["pair_of_row"], r["row_of_pair"]
    xp = M.permute(L.x, por, k, row_of_pair=rop)
    x4 = M.fp4_quantize(xp, off, fmt=fmt)
    a, z, err = M.fp4_linear(x4, off, L.w1, fmt=fmt, act="swiglu", w_scale=L.t1, save_z=True)
    a4 = M.fp4_quantize(a, off, fmt=fmt)
    y, _, _ = M.fp4_linear(a4, off, L.w2, fmt=fmt, w_scale=L.t2, err=err)
    dout = torch.randn((T, d), generator=torch.Generator().manual_seed(9)).to(BF).to(DEV)
    dy = M.permute(dout, por, k, scale=probs.reshape(-1), row_of_pair=rop)
    _, dprobs = M.unpermute(y, rop, T, k, dO=dout, combine=False)
    _, da, dW2, _, _ = M.fp4_linear_bwd(dy, a, off, L.w2b, fmt=fmt, w_scale=L.t2, err=err)
    dz, dxp, dW1, _, _ = M.fp4_linear_bwd(da, xp, off, L.w1b, fmt=fmt, act="swiglu", z=z, w_scale=L.t1, err=err)
    dx, _ = M.unpermute(dxp, rop, T, k)
    dloss = torch.tensor([0.1, 0.01], device=DEV)
    dlogits = M.router_loss_bwd(L.logits, idx, loss, dloss)
    M.router_select_bwd(L.logits, idx, probs, dprobs, score="sigmoid", scale=2.5, dlogits=dlogits, accumulate=True)
    torch.cuda.synchronize()
    assert int(err) == 0
    # float64, from the values that each product took
    o = off.cpu().tolist()
    w1b = _f64(M.fp4_dequantize(L.w1b, fmt=fmt, scale=L.t1, dtype=F32))
    w2b = _f64(M.fp4_dequantize(L.w2b, fmt=fmt, scale=L.t2, dtype=F32))
    scale = lambda v: F.tensor_scale(v) if fmt == "nvfp4" else 1.0  # noqa: E731
    g2, g1 = _f64(dy), _f64(dz)
    g2h, g1h = _held(g2, fmt, scale(g2)), _held(g1, fmt, scale(g1))
    zz, dA = _f64(z), _f64(da)
    sg = 1 / (1 + np.exp(-zz[:, 0::2]))
    ref_dz = np.empty_like(zz)
    ref_dz[:, 0::2] = dA * zz[:, 1::2] * sg * (1 + zz[:, 0::2] * (1 - sg))
    ref_dz[:, 1::2] = dA * zz[:, 0::2] * sg
    _close(g1, ref_dz, "dz", 0.003)
    ref_da, ref_dx = np.zeros_like(dA), np.zeros((o[-1], d))
    rW1, rW2 = np.zeros((E, d, 2 * n)), np.zeros((E, n, d))
    for e in range(E):
        i, j = o[e], o[e + 1]
        ref_da[i:j], ref_dx[i:j] = g2h[i:j] @ w2b[e].T, g1h[i:j] @ w1b[e].T
        rW1[e], rW2[e] = _f64(xp)[i:j].T @ g1[i:j], _f64(a)[i:j].T @ g2[i:j]
    _close(dA, ref_da, "da", 0.003)
    _close(_f64(dxp), ref_dx, "dx of the rows", 0.003)
    _close(_f64(dW1), rW1, "dW1", 0.003)
    _close(_f64(dW2), rW2, "dW2", 0.003)
    ref_dp = np.zeros((T, k))
    rows = rop.cpu().numpy().reshape(T, k)
    for t in range(T):
        ref_dp[t] = _f64(y)[rows[t]] @ _f64(dout)[t]
    _close(_f64(dprobs), ref_dp, "dprobs", 1e-5)
    ref_dl = S.router_select_bwd(_f64(L.logits), idx.cpu().numpy(), ref_dp, "sigmoid", True, 2.5)
    ref_dl = ref_dl + O.router_loss_bwd(_f64(L.logits), idx.cpu().numpy(), _f64(dloss), None, None)
    _close(_f64(dlogits), ref_dl, "dlogits", 1e-5)
    # the whole layer's gradient is near the bf16 layer's: 4 bits of each operand
    # are off by a tenth of its 2-norm, three products deep
    assert np.isfinite(_f64(dx)).all()
