"""The products in 4 bits against float64 products of the values their
operands stand for (moe_fp4_linear, moe_fp4_linear_bwd)."""
import numpy as np
import pytest
import torch

import dropless_grouped_gemm_gb300 as M
from oracle import fp4 as O

pytestmark = pytest.mark.gpu
BF, F32, U8, I32, F64 = torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.float64
DEV = "cuda"
FMT = ["nvfp4", "mxfp4"]
ACTS = ["none", "relu", "silu", "gelu", "srelu", "swiglu", "geglu"]


def _gated(act):
    return act in ("swiglu", "geglu")


def _act(z, act):
    g = z[:, 0::2] if _gated(act) else z
    if act in ("silu", "swiglu"):
        p = g * torch.sigmoid(g)
    elif act in ("gelu", "geglu"):
        p = 0.5 * g * (1 + torch.tanh((2 / np.pi) ** 0.5 * (g + 0.044715 * g ** 3)))
    elif act == "relu":
        p = g.clamp(min=0)
    elif act == "srelu":
        p = g.clamp(min=0) ** 2
    else:
        p = g
    return p * z[:, 1::2] if _gated(act) else p


class Case:
    """Operands of one product, quantised by the framework, and the values in
    64 bits that they stand for (the quantisers have tests of their own)."""

    def __init__(self, offsets, K, N, fmt, seed=0, extra=0, scaled=True, dense=False):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.offsets, self.K, self.N, self.fmt, self.E = offsets, K, N, fmt, len(offsets) - 1
        self.last = offsets[-1]
        self.rows = self.last + extra
        self.x = torch.randn((self.rows, K), generator=g, device=DEV).to(BF)
        self.W = (0.05 * torch.randn((self.E, N, K), generator=g, device=DEV)).to(BF)
        self.off = None if dense else torch.tensor(offsets, dtype=I32, device=DEV)
        nv = fmt == "nvfp4" and scaled
        self.at = torch.tensor([0.5], device=DEV) if nv else None
        self.wt = M.fp4_tensor_scale(self.W, per_expert=True) if nv else None
        self.a = M.fp4_quantize(self.x, self.off, fmt=fmt, scale=self.at)
        self.w = M.fp4_quantize_weights(self.W, fmt=fmt, along="cols", scale=self.wt)
        self.bias = (0.5 * torch.randn((self.E, N), generator=g, device=DEV)).to(BF)
        self.xv = torch.zeros((self.rows, K), device=DEV)
        M.fp4_dequantize(self.a, self.off, fmt=fmt, scale=self.at, out=self.xv)
        self.wv = M.fp4_dequantize(self.w, fmt=fmt, scale=self.wt, dtype=F32)

    def spans(self):
        return [(e, a, b) for e, (a, b) in enumerate(zip(self.offsets[:-1], self.offsets[1:])) if b > a]

    def z64(self, bias):
        """z and the sum of its terms' magnitudes (the rounding's scale)."""
        z = torch.zeros((self.last, self.N), dtype=F64, device=DEV)
        mag = torch.zeros_like(z)
        for e, a, b in self.spans():
            x, w = self.xv[a:b].double(), self.wv[e].double()
            z[a:b], mag[a:b] = x @ w.T, x.abs() @ w.abs().T
            if bias:
                z[a:b] += self.bias[e].double()
                mag[a:b] += self.bias[e].double().abs()
        return z, mag

    def tol_z(self, mag):
        """Each of K / 64 MMAs of a chain, each of up to 8 parts, and bias and
        scale round a sum of magnitude at most mag, by at most 2^-22 of it
        (the tensor cores' accumulation is not a full float32 addition)."""
        return (self.K / 64 + 10) * 2.0 ** -22 * mag

    def run(self, **kw):
        return M.fp4_linear(self.a, self.off, self.w, fmt=self.fmt, a_scale=self.at, w_scale=self.wt, **kw)


def _slope(act):
    """How much of an error of z reaches the output, per unit of |z| + 1."""
    return 1.2 if act in ("none", "relu", "silu", "gelu") else 2.5


def _check(c, act="none", bias=True, residual=False, out_dtype=BF, save_z=False):
    n_out = c.N // 2 if _gated(act) else c.N
    res = torch.randn((c.rows, n_out), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(BF) if residual else None
    out = torch.full((c.rows, n_out), 3.0, dtype=out_dtype, device=DEV)
    z = torch.full((c.rows, c.N), 5.0, dtype=BF, device=DEV) if save_z else None
    err = torch.zeros(1, dtype=I32, device=DEV)
    got, _, _ = c.run(act=act, bias=c.bias if bias else None, residual=res, out=out, z=z, err=err)
    torch.cuda.synchronize()
    assert got is out and int(err) == 0
    z64, mag = c.z64(bias)
    tz = c.tol_z(mag)
    ref = _act(z64, act)
    # the activation's own float32 arithmetic: 2^-19 of z's magnitude (exp and
    # an approximate division, a few units each, times up to z)
    big = z64.abs() + 1
    if _gated(act):
        pair = lambda t: t[:, 0::2] + t[:, 1::2]
        tol = _slope(act) * (pair(tz) + pair(tz) * pair(big)) + 2.0 ** -19 * big[:, 0::2] * big[:, 1::2]
    else:
        tol = _slope(act) * tz * (big if act == "srelu" else 1) + 2.0 ** -19 * (big ** 2 if act == "srelu" else big)
    if residual:
        ref = ref + res[:c.last].double()
        tol = tol + 2.0 ** -23 * res[:c.last].double().abs()
    if out_dtype is BF:
        tol = tol + 2.0 ** -8 * ref.abs()
    bad = (out[:c.last].double() - ref).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), float((out[:c.last].double() - ref).abs().max()))
    assert (out[c.last:] == 3).all()
    if save_z:
        assert ((z[:c.last].double() - z64).abs() <= tz + 2.0 ** -8 * z64.abs()).all()
        assert (z[c.last:] == 5).all()


# few rows: every split, odd tiles (a second 64 rows of a 128-row scale tile), N
# that ends inside a tile, K that ends inside a stage and inside a chunk
FEW = [([0, 1], 64, 64), ([0, 1], 7168, 128), ([0, 16], 2048, 512), ([0, 17], 576, 192), ([0, 64], 1088, 320),
       ([0, 65], 512, 128), ([0, 128], 320, 64), ([0, 200], 1024, 448), ([0, 1, 1, 2, 30], 448, 256),
       ([0, 0, 70, 70, 137, 400], 704, 128), ([0, 0], 128, 128), ([0, 33, 33], 4096, 192)]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("offsets,K,N", FEW)
@pytest.mark.parametrize("dense", [False, True])
def test_few_rows(fmt, offsets, K, N, dense):
    if dense and len(offsets) > 2:
        pytest.skip("one expert")
    c = Case(offsets, K, N, fmt, extra=0 if dense else 5, dense=dense)
    _check(c, out_dtype=F32)
    _check(c, act="swiglu" if N % 128 == 0 else "silu", residual=True, save_z=True)


@pytest.mark.parametrize("split", [1, 2, 4, 8])
def test_every_split(split):
    """Sizes for which the kernel choice takes each split, found by asking it."""
    sizes = [(m, k, n) for k in (512, 1024, 2048, 4096, 7168) for n in (128, 512, 1152, 2048, 4096, 8192) for m in (1, 16, 40, 64, 100, 200)]
    takes = [x for x in sizes if M.fp4_linear_plan(1, *x, False) == (64, split)]
    assert takes
    for m, k, n in (takes[0], takes[len(takes) // 2], takes[-1]):
        for fmt in FMT:
            _check(Case([0, m], k, n, fmt, dense=True), act="swiglu", residual=True)


# many rows: the pairs' kernel
MANY = [([0, 2048], 2048, 2048), ([0, 9000], 1088, 1088), ([0, 700, 700, 1999, 12000], 960, 1344), ([0, 1, 9000, 9001], 2048, 1024),
        ([0, 0, 16383], 2048, 1088)]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("offsets,K,N", MANY)
def test_many_rows(fmt, offsets, K, N):
    c = Case(offsets, K, N, fmt, extra=7)
    assert M.fp4_linear_plan(c.E, c.rows, K, N, True)[0] == 0
    _check(c, out_dtype=F32)
    _check(c, act="geglu" if N % 128 == 0 else "gelu", residual=True, save_z=True)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("offsets,K,N", [([0, 40], 512, 256), ([0, 3000, 8192], 512, 2048)])
def test_activations(fmt, act, offsets, K, N):
    c = Case(offsets, K, N, fmt)
    _check(c, act=act, out_dtype=F32)
    _check(c, act=act, bias=False, residual=True)


def test_without_tensor_scales():
    for offsets in ([0, 20], [0, 8192]):
        _check(Case(offsets, 512, 2048, "nvfp4", scaled=False), out_dtype=F32)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("act", ["none", "srelu", "swiglu", "geglu"])
@pytest.mark.parametrize("offsets,K,N", [([0, 1], 512, 128), ([0, 70, 70, 137], 512, 384), ([0, 300], 2048, 1152), ([0, 2000, 2000, 12000], 512, 1152)])
def test_four_bit_outputs(fmt, act, offsets, K, N):
    c = Case(offsets, K, N, fmt, extra=4)
    n_out = N // 2 if _gated(act) else N
    t = torch.tensor([0.25], device=DEV) if fmt == "nvfp4" else None
    poison = (torch.full((c.rows, n_out // 2), 0xAB, dtype=U8, device=DEV),
              torch.full((M.fp4_scale_bytes(c.rows, c.E, n_out, fmt),), 0xCD, dtype=U8, device=DEV))
    (q, s), _, err = c.run(act=act, bias=c.bias, out=poison, out_scale=t)
    full, _, _ = c.run(act=act, bias=c.bias, out_dtype=F32)
    assert int(err) == 0
    # the codes of the float32 outputs, but where a quotient lies within 2^-22 of
    # a border (the same float32 values: a reciprocal's and a product's rounding)
    v = full[:c.last].double().cpu().numpy()
    tf = 1.0 if t is None else float(t)
    code, byte = O.quantize(v, fmt, tf)
    at = O.scale_place(offsets, n_out, fmt)
    sb = s.cpu().numpy()
    np.testing.assert_array_equal(sb[at], byte)
    d = np.repeat(O.scale_values(byte, fmt) * tf, O.BLOCK[fmt], -1)
    with np.errstate(divide="ignore", invalid="ignore"):
        u = np.abs(v) / d
    halves = (O.MAGNITUDES[1:] + O.MAGNITUDES[:-1]) / 2
    near = (np.abs(u[..., None] / halves - 1) < 2.0 ** -21).any(-1)
    got = O.unpack(q[:c.last].cpu().numpy())
    assert ((O.code_values(got) == O.code_values(code)) | near).all()
    free = np.ones(sb.size, bool)
    free[at.reshape(-1)] = False
    assert (sb[free] == 0xCD).all() and (q[c.last:] == 0xAB).all()


@pytest.mark.parametrize("rows", [30, 9000])
def test_a_nan_stays_in_its_row(rows):
    for fmt in FMT:
        c = Case([0, rows // 3, rows], 512, 2048, fmt)
        clean, _, _ = c.run()
        x = c.x.clone()
        x[5, 100], x[rows - 1, 0] = float("nan"), float("inf")
        a = M.fp4_quantize(x, c.off, fmt=fmt, scale=c.at)
        out, _, _ = M.fp4_linear(a, c.off, c.w, fmt=fmt, a_scale=c.at, w_scale=c.wt)
        assert torch.isnan(out[5]).all() and torch.isnan(out[rows - 1]).all()
        keep = torch.ones(rows, dtype=torch.bool)
        keep[5] = keep[rows - 1] = False
        assert torch.equal(out[keep.to(DEV)], clean[keep.to(DEV)])


def test_what_lies_behind_the_rows_does_not_matter():
    """Rows, scales and codes of no expert hold NaN scales and any codes."""
    for rows, fmt in ((40, "nvfp4"), (40, "mxfp4"), (9000, "nvfp4"), (9000, "mxfp4")):
        c = Case([0, rows // 2, rows], 576, 1088, fmt)
        ref, _, _ = c.run()
        total = rows + 300
        s = torch.full((M.fp4_scale_bytes(total, 2, c.K, fmt),), 0x7F if fmt == "nvfp4" else 0xFF, dtype=U8, device=DEV)
        q = torch.full((total, c.K // 2), 0x77, dtype=U8, device=DEV)
        x = torch.full((total, c.K), float("nan"), dtype=BF, device=DEV)
        x[:rows] = c.x
        a = M.fp4_quantize(x, c.off, fmt=fmt, scale=c.at, out=(q, s))
        out, _, err = M.fp4_linear(a, c.off, c.w, fmt=fmt, a_scale=c.at, w_scale=c.wt)
        assert int(err) == 0 and torch.equal(out[:rows], ref)


def test_reruns_and_residual_in_place():
    for rows in (48, 9000):
        c = Case([0, rows], 1024, 1024, "nvfp4")
        one = c.run(bias=c.bias)[0]
        assert torch.equal(one, c.run(bias=c.bias)[0])
        res = torch.randn_like(one)
        ref = c.run(residual=res)[0]
        buf = res.clone()
        assert torch.equal(c.run(residual=buf, out=buf)[0], ref)


def test_bad_offsets_are_corrected_and_reported():
    for rows in (60, 9000):
        x = torch.randn(rows, 256, device=DEV).to(BF)
        w = M.fp4_quantize_weights(0.1 * torch.randn(3, 1024, 256, device=DEV).to(BF), along="cols")
        for off, safe in (([0, rows, rows // 2, rows], [0, rows, rows, rows]), ([0, -3, 7, rows + 9], [0, 0, 7, rows])):
            o, s = (torch.tensor(v, dtype=I32, device=DEV) for v in (off, safe))
            err = torch.zeros(1, dtype=I32, device=DEV)
            a, b = M.fp4_quantize(x, o), M.fp4_quantize(x, s)
            out, _, _ = M.fp4_linear(a, o, w, err=err)
            ref, _, e2 = M.fp4_linear(b, s, w)
            assert int(err) == M.DEV_BAD_OFFSETS and int(e2) == 0 and torch.equal(out, ref)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("offsets", [[0, 30], [0, 0, 70, 137], [5, 70, 70, 600]])
def test_backward_does_not_see_other_rows(fmt, act, offsets):
    """Large finite values, infinities and NaN in the rows of no expert, in
    front of the first one and behind the last, in dout, z, a and dz's buffer:
    the gradients of the experts' rows stay what they are with zeros there."""
    K, N, rows = 192, 256, offsets[-1] + 40
    g = torch.Generator(device=DEV).manual_seed(8)
    E, n_out = len(offsets) - 1, N // 2 if _gated(act) else N
    off = torch.tensor(offsets, dtype=I32, device=DEV)
    wt = M.fp4_quantize_weights(0.1 * torch.randn((E, K, N), generator=g, device=DEV).to(BF), fmt=fmt, along="cols")
    a, z, dout = (torch.randn((rows, n), generator=g, device=DEV).to(BF) for n in (K, N, n_out))
    outs = []
    for other in (0.0, 1e30, float("inf"), float("nan")):
        x = [t.clone() for t in (a, z, dout, torch.zeros(rows, N, dtype=BF, device=DEV))]
        for t in x:
            t[:offsets[0]] = other
            t[offsets[-1]:] = other
        err = torch.zeros(1, dtype=I32, device=DEV)
        dz, da, dB, db, _ = M.fp4_linear_bwd(x[2], x[0], off, wt, fmt=fmt, act=act, z=x[1] if act != "none" else None,
                                             bias=True, dz=x[3] if act != "none" else None, err=err)
        mine = slice(offsets[0], offsets[-1])
        outs.append((dz[mine], da[mine], dB, db))
    for o in outs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(o, outs[0]))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("act", ["none", "silu", "srelu", "swiglu", "geglu"])
@pytest.mark.parametrize("offsets,K,N,layout", [([0, 30], 192, 256, "kn"), ([0, 0, 70, 137], 320, 128, "nk"), ([0, 1500, 1500, 9000], 1024, 1152, "kn")])
def test_backward(fmt, act, offsets, K, N, layout):
    c = Case(offsets, K, N, fmt, extra=3)
    g = torch.Generator(device=DEV).manual_seed(4)
    n_out = N // 2 if _gated(act) else N
    W = c.W.transpose(1, 2).contiguous()                              # [E, K, N]
    wt_t = M.fp4_tensor_scale(W, per_expert=True) if fmt == "nvfp4" else None
    wt = M.fp4_quantize_weights(W, fmt=fmt, along="cols", scale=wt_t)
    z = torch.randn((c.rows, N), generator=g, device=DEV).to(BF) if act != "none" else None
    dout = (1e-4 * torch.randn((c.rows, n_out), generator=g, device=DEV)).to(BF)
    dout[c.last:] = 0
    if z is not None:
        z[c.last:] = 0
    da = torch.full((c.rows, K), 9.0, dtype=BF, device=DEV)
    dz, da, dB, db, err = M.fp4_linear_bwd(dout, c.x, c.off, wt, fmt=fmt, act=act, z=z, bias=True, w_scale=wt_t,
                                           b_layout=layout, da=da)
    B = W if layout == "kn" else c.W
    dz1, _, dB1, db1, _ = M.grouped_linear_bwd(dout, c.x, c.off, B, act=act, z=z, bias=True, b_layout=layout)
    assert int(err) == 0
    assert torch.equal(dz[:c.last], dz1[:c.last]) and torch.equal(dB, dB1) and torch.equal(db, db1)
    # the data gradient: a float64 product of the oracle's 4-bit dz
    d = dz.float().cpu().numpy().astype(np.float64)
    t = O.tensor_scale(d[:c.last]) if fmt == "nvfp4" else 1.0          # (dz behind the rows is not written)
    dv = torch.from_numpy(O.values(*O.quantize(d, fmt, t), fmt, t)).to(DEV)
    wv = M.fp4_dequantize(wt, fmt=fmt, scale=wt_t, dtype=F32).double()
    for e, a, b in c.spans():
        ref, mag = dv[a:b] @ wv[e].T, dv[a:b].abs() @ wv[e].abs().T
        assert ((da[a:b].double() - ref).abs() <= (N / 64 + 10) * 2.0 ** -22 * mag + 2.0 ** -8 * ref.abs()).all()
    assert (da[c.last:] == 9).all()
    # accumulated weight gradients
    dB2, db2 = dB.clone(), db.clone()
    M.fp4_linear_bwd(dout, c.x, c.off, wt, fmt=fmt, act=act, z=z, bias=True, w_scale=wt_t, b_layout=layout, dB=dB2, dbias=db2,
                     accumulate_dw=True)
    dB3, db3 = dB1.clone(), db1.clone()
    M.grouped_linear_bwd(dout, c.x, c.off, B, act=act, z=z, bias=True, b_layout=layout, dB=dB3, dbias=db3, accumulate_dw=True)
    assert torch.equal(dB2, dB3) and torch.equal(db2, db3)


def test_gradient_against_differences():
    """With the codes held, the product is linear in a's values: da of a dense
    gradient equals the product's differences in each direction."""
    c = Case([0, 8], 64, 128, "mxfp4")
    W = c.W.transpose(1, 2).contiguous()
    # weights whose two copies hold the same values: powers of two below 6
    W = torch.sign(W) * 2.0 ** torch.randint(-1, 3, W.shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(3))
    W = W.to(BF)
    w, wt = M.fp4_quantize_weights(W, fmt="mxfp4", along="rows"), M.fp4_quantize_weights(W, fmt="mxfp4", along="cols")
    x = torch.randint(-3, 4, (8, 64), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(BF)
    dout = torch.randint(-2, 3, (8, 128), device=DEV, generator=torch.Generator(device=DEV).manual_seed(2)).to(BF)
    # (a 4 in every block keeps scales and so all small whole numbers as they are)
    x[:, ::32] = 4
    dout[:, ::32] = 4
    _, da, _, _, _ = M.fp4_linear_bwd(dout, x, None, wt, fmt="mxfp4")
    f = lambda v: float((M.fp4_linear(M.fp4_quantize(v, fmt="mxfp4"), None, w, fmt="mxfp4", out_dtype=F32)[0].double() * dout.double()).sum())
    for r, k in ((0, 1), (3, 17), (7, 63), (5, 33)):
        hi, lo = x.clone(), x.clone()
        hi[r, k], lo[r, k] = 2, 0
        # small whole numbers and their halves: everything is exact
        assert (f(hi) - f(lo)) / 2 == float(da[r, k])


def test_in_a_graph_and_on_another_stream():
    c = Case([0, 30, 90], 512, 512, "nvfp4")
    big = Case([0, 2000, 9000], 512, 1024, "nvfp4")
    for k in (c, big):
        ref = k.run(act="swiglu", bias=k.bias)[0].clone()
        out = torch.zeros_like(ref)
        err = torch.zeros(1, dtype=I32, device=DEV)
        x = k.x.clone()
        a = tuple(torch.zeros_like(t) for t in k.a)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        y = M.fp4_linear(M.fp4_quantize(x, k.off, scale=k.at, stream=s), k.off, k.w, act="swiglu", bias=k.bias, a_scale=k.at,
                         w_scale=k.wt, stream=s)[0]
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(y, ref)
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                M.fp4_quantize(x, k.off, scale=k.at, out=a, err=err)
                M.fp4_linear(a, k.off, k.w, act="swiglu", bias=k.bias, a_scale=k.at, w_scale=k.wt, out=out, err=err)
        torch.cuda.synchronize()
        x.zero_()
        g.replay()
        torch.cuda.synchronize()
        x.copy_(k.x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and int(err) == 0
