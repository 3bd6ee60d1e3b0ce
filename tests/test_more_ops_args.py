"""What the choice by scores and the products in 4 bits refuse, on the host and
before anything is enqueued: the C entry points' return codes, and the
binding's checks against stand-ins for CUDA tensors (no GPU needed)."""
import ctypes

import pytest
import torch

import dropless_grouped_gemm_gb300 as M
from dropless_grouped_gemm_gb300 import build as B
from test_binding_checks import BF, F32, I32, U8, Fake, Lib, _refused

NULL, ALIGN, SIZE, ARG, WS = -1, -2, -3, -4, -6
vp = ctypes.c_void_p
P = vp(16)          # an aligned address that nothing reads


@pytest.fixture(scope="module")
def L():
    B.build()
    return M.lib()


def _select(L, **kw):
    a = dict(z=P, lt=0, T=4, E=8, k=2, score=0, bias=P, g=1, tg=1, gb=1, rn=1, sc=1.0, idx=P, pr=P)
    a.update(kw)
    return L.moe_router_select(a["z"], a["lt"], a["T"], a["E"], a["k"], a["score"], a["bias"], a["g"], a["tg"], a["gb"], a["rn"],
                               a["sc"], a["idx"], a["pr"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), SIZE), (dict(T=(1 << 30) + 1), SIZE), (dict(E=0), SIZE), (dict(E=1025), SIZE), (dict(k=0), SIZE), (dict(k=9), SIZE),
    (dict(E=64, k=33), SIZE), (dict(g=0), SIZE), (dict(g=3), SIZE), (dict(E=66, g=33), SIZE), (dict(g=4, tg=5), SIZE),
    (dict(g=4, tg=0), SIZE), (dict(g=8, tg=1), SIZE), (dict(g=4, tg=1, k=3), SIZE), (dict(g=8, tg=8, gb=2), SIZE), (dict(gb=3), SIZE),
    (dict(gb=0), SIZE), (dict(score=2), ARG), (dict(rn=2), ARG), (dict(sc=0.0), ARG), (dict(sc=-1.0), ARG),
    (dict(sc=float("inf")), ARG), (dict(sc=float("nan")), ARG), (dict(lt=2), ARG), (dict(z=None), NULL), (dict(idx=None), NULL),
    (dict(pr=None), NULL), (dict(z=vp(18)), ALIGN), (dict(z=vp(17), lt=1), ALIGN), (dict(bias=vp(18)), ALIGN), (dict(pr=vp(2)), ALIGN),
    (dict(T=0, z=None, idx=None, pr=None), 0)])
def test_router_select(L, kw, rc):
    assert _select(L, **kw) == rc


def _select_bwd(L, **kw):
    a = dict(z=P, lt=0, idx=P, pr=P, dp=P, T=4, E=8, k=2, score=0, rn=1, sc=1.0, acc=0, out=P, ot=0)
    a.update(kw)
    return L.moe_router_select_bwd(a["z"], a["lt"], a["idx"], a["pr"], a["dp"], a["T"], a["E"], a["k"], a["score"], a["rn"], a["sc"],
                                   a["acc"], a["out"], a["ot"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(E=0), SIZE), (dict(k=9), SIZE), (dict(score=-1), ARG), (dict(acc=2), ARG), (dict(ot=2), ARG), (dict(sc=0.0), ARG),
    (dict(z=None), NULL), (dict(idx=None), NULL), (dict(pr=None), NULL), (dict(dp=None), NULL), (dict(out=None), NULL),
    (dict(out=vp(18)), ALIGN), (dict(out=vp(17), ot=1), ALIGN), (dict(dp=vp(6)), ALIGN), (dict(T=0), 0)])
def test_router_select_bwd(L, kw, rc):
    assert _select_bwd(L, **kw) == rc


def test_sizes(L):
    f = L.moe_fp4_scale_bytes
    assert f(300, 4, 192, 0) == (2 + 4) * 3 * 512 and f(300, 4, 192, 1) == (2 + 4) * 2 * 512
    assert f(0, 1, 64, 0) == 512 and f(300, 0, 192, 0) == 0 and f(300, 4, 100, 0) == 0 and f(-1, 4, 192, 0) == 0
    assert f(300, 4, 192, 2) == 0 and f(1 << 33, 1, 8192, 0) == 0
    for a in ((300, 4, 192), (1, 1, 64), (129, 7, 7168)):
        assert M.fp4_scale_bytes(*a, "nvfp4") == f(*a, 0) and M.fp4_scale_bytes(*a, "mxfp4") == f(*a, 1)
    w = L.moe_fp4_linear_bwd_workspace_size
    assert w(4, 300, 192, 0) >= 300 * 96 + f(300, 4, 192, 0) and w(4, 300, 100, 0) == 0 and w(0, 300, 192, 0) == 0
    assert M.fp4_linear_bwd_workspace_size(4, 300, 192, "mxfp4") == w(4, 300, 192, 1)


def test_quantisers(L):
    t = L.moe_fp4_tensor_scale
    assert t(P, 0, 64, P, None) == SIZE and t(P, 1, 63, P, None) == SIZE and t(P, 1, -64, P, None) == SIZE
    assert t(P, 1, 64, None, None) == NULL and t(None, 1, 64, P, None) == NULL and t(vp(8), 1, 64, P, None) == ALIGN
    q = lambda src=P, off=P, E=2, rows=8, K=64, f=0, t=P, qq=P, s=P, err=P: L.moe_fp4_quantize(src, off, E, rows, K, f, t, qq, s, err, None)  # noqa: E731
    for kw, rc in ((dict(E=0), SIZE), (dict(rows=-1), SIZE), (dict(K=96), SIZE), (dict(K=(1 << 23) + 64), SIZE), (dict(off=None, rows=9), SIZE),
                   (dict(f=2), ARG), (dict(f=1), ARG), (dict(src=None), NULL), (dict(qq=None), NULL), (dict(s=None), NULL), (dict(err=None), NULL),
                   (dict(src=vp(8)), ALIGN), (dict(qq=vp(8)), ALIGN), (dict(s=vp(8)), ALIGN), (dict(t=vp(2)), ALIGN), (dict(rows=0), 0)):
        assert q(**kw) == rc, kw
    p = lambda src=P, rop=P, por=P, off=P, E=2, T=4, k=2, K=64, M_=8, f=0, t=P, qq=P, s=P, err=P: L.moe_fp4_permute(src, rop, por, off, E, T, k, K, M_, f, t, qq, s, err, None)  # noqa: E731
    for kw, rc in ((dict(T=-1), SIZE), (dict(k=0), SIZE), (dict(T=1 << 28, k=8), SIZE), (dict(K=32), SIZE), (dict(M_=-1), SIZE), (dict(f=1), ARG),
                   (dict(por=None), NULL), (dict(off=None), NULL), (dict(src=None), NULL), (dict(src=vp(4)), ALIGN), (dict(M_=0), 0)):
        assert p(**kw) == rc, kw
    w = lambda W=P, E=2, r=64, c=64, al=1, f=0, t=P, qq=P, s=P: L.moe_fp4_quantize_weights(W, E, r, c, al, f, t, qq, s, None)  # noqa: E731
    for kw, rc in ((dict(E=0), SIZE), (dict(r=0), SIZE), (dict(r=96), SIZE), (dict(c=96), SIZE), (dict(al=2), ARG), (dict(f=1), ARG), (dict(f=7, t=None), ARG),
                   (dict(W=None), NULL), (dict(W=vp(2)), ALIGN), (dict(s=vp(4)), ALIGN)):
        assert w(**kw) == rc, kw
    d = lambda q=P, s=P, off=P, E=2, rows=8, K=64, f=0, t=P, pe=0, o=P, ty=1, err=P: L.moe_fp4_dequantize(q, s, off, E, rows, K, f, t, pe, o, ty, err, None)  # noqa: E731
    for kw, rc in ((dict(E=0), SIZE), (dict(rows=1 << 32), SIZE), (dict(off=None, rows=9), SIZE), (dict(ty=2), ARG), (dict(pe=2), ARG), (dict(f=1), ARG),
                   (dict(q=None), NULL), (dict(o=None), NULL), (dict(o=vp(8)), ALIGN), (dict(rows=0), 0)):
        assert d(**kw) == rc, kw


def _linear(L, **kw):
    a = dict(aq=P, as_=P, at=P, off=P, E=2, M=8, K=64, N=128, wq=P, ws=P, wt=P, f=0, bias=P, act=3, res=P, z=P, out=P, ot=1, os=None, tt=None, err=P)
    a.update(kw)
    return L.moe_fp4_linear(a["aq"], a["as_"], a["at"], a["off"], a["E"], a["M"], a["K"], a["N"], a["wq"], a["ws"], a["wt"], a["f"], a["bias"], a["act"],
                            a["res"], a["z"], a["out"], a["ot"], a["os"], a["tt"], a["err"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(E=0), SIZE), (dict(E=1025), SIZE), (dict(M=-1), SIZE), (dict(K=96), SIZE), (dict(N=32), SIZE), (dict(off=None), SIZE),
    (dict(N=(1 << 23) + 64), SIZE), (dict(act=0, N=64, ot=2, os=P), SIZE),        # 32 outputs are no chunk's row
    (dict(act=7), ARG), (dict(ot=3), ARG), (dict(f=2), ARG), (dict(f=1), ARG), (dict(os=P), ARG), (dict(tt=P), ARG),
    (dict(aq=None), NULL), (dict(as_=None), NULL), (dict(wq=None), NULL), (dict(ws=None), NULL), (dict(out=None), NULL), (dict(err=None), NULL),
    (dict(ot=2), NULL), (dict(aq=vp(8)), ALIGN), (dict(as_=vp(8)), ALIGN), (dict(wq=vp(8)), ALIGN), (dict(ws=vp(8)), ALIGN), (dict(bias=vp(8)), ALIGN),
    (dict(res=vp(8)), ALIGN), (dict(z=vp(8)), ALIGN), (dict(out=vp(8)), ALIGN), (dict(wt=vp(2)), ALIGN), (dict(ot=2, os=vp(8)), ALIGN), (dict(M=0), 0)])
def test_linear(L, kw, rc):
    assert _linear(L, **kw) == rc


def _linear_bwd(L, **kw):
    a = dict(dout=P, z=P, a=P, off=P, E=2, M=8, K=64, N=128, wq=P, ws=P, wt=P, f=0, lay=0, act=0, fl=0, dz=P, da=P, dB=P, db=P, w=P, wb=1 << 20, err=P)
    a.update(kw)
    return L.moe_fp4_linear_bwd(a["dout"], a["z"], a["a"], a["off"], a["E"], a["M"], a["K"], a["N"], a["wq"], a["ws"], a["wt"], a["f"], a["lay"], a["act"],
                                a["fl"], a["dz"], a["da"], a["dB"], a["db"], a["w"], a["wb"], a["err"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(K=32), SIZE), (dict(N=96), SIZE), (dict(off=None), SIZE), (dict(act=9), ARG), (dict(lay=2), ARG), (dict(fl=1), ARG), (dict(f=1), ARG),
    (dict(f=5, wt=None), ARG), (dict(wq=None), NULL), (dict(ws=None), NULL), (dict(dout=None), NULL), (dict(z=None), NULL), (dict(dz=None), NULL),
    (dict(a=None), NULL), (dict(err=None), NULL), (dict(w=None), NULL), (dict(w=vp(8)), ALIGN), (dict(wb=64), WS), (dict(da=vp(8)), ALIGN),
    (dict(wq=vp(8)), ALIGN), (dict(db=vp(8)), ALIGN)])
def test_linear_bwd(L, kw, rc):
    assert _linear_bwd(L, **kw) == rc


def test_plan_arguments(L):
    plan = (ctypes.c_int * 2)()
    r = ctypes.byref(plan)
    assert L.moe_fp4_linear_plan(1, 8, 96, 64, 0, r) == SIZE and L.moe_fp4_linear_plan(1, 0, 64, 64, 0, r) == SIZE
    assert L.moe_fp4_linear_plan(2, 8, 64, 64, 0, r) == SIZE and L.moe_fp4_linear_plan(1, 8, 64, 64, 2, r) == ARG
    assert L.moe_fp4_linear_plan(1, 8, 64, 64, 0, None) == NULL


# ------------------------------------------------ the binding

@pytest.fixture
def FL(monkeypatch):
    lib = Lib()
    monkeypatch.setattr(M, "lib", lambda: lib)
    monkeypatch.setattr(M, "_stream", lambda s=None: 0)
    monkeypatch.setattr(M, "_err_word", lambda err, dev, stream=None: err or Fake(1, I32))
    monkeypatch.setattr(M, "_empty", lambda shape, dtype, dev, stream=None: Fake(shape, dtype))
    monkeypatch.setattr(M, "_scratch", lambda n, dev, stream=None: Fake(n, U8))
    return lib


def _pair(rows, K, E=1, fmt="nvfp4", lead=None):
    return Fake((rows, K // 2) if lead is None else (lead, rows // lead, K // 2), U8), Fake(M.fp4_scale_bytes(rows, E, K, fmt), U8)


@pytest.mark.parametrize("bad", [
    dict(k=2, score="tanh"), dict(k=2, bias=Fake(7, F32)), dict(k=2, bias=Fake(8, BF)), dict(k=2, topk_idx=Fake((10, 3), I32)),
    dict(k=2, probs=Fake((10, 2), BF)), dict(k=2, probs=Fake((10, 2), F32, contiguous=False))])
def test_select_refuses(FL, bad):
    _refused(FL, lambda: M.router_select(Fake((10, 8), F32), **bad))
    _refused(FL, lambda: M.router_select(Fake((10, 8), torch.float16), 2))
    _refused(FL, lambda: M.router_select(Fake((10, 8), F32, is_cuda=False), 2))


def test_select_bwd_refuses(FL):
    z, i, p = Fake((10, 8), F32), Fake((10, 2), I32), Fake((10, 2), F32)
    for call in (lambda: M.router_select_bwd(z, Fake((9, 2), I32), p, p), lambda: M.router_select_bwd(z, i, Fake((10, 3), F32), p),
                 lambda: M.router_select_bwd(z, i, p, None), lambda: M.router_select_bwd(z, i, p, p, accumulate=True),
                 lambda: M.router_select_bwd(z, i, p, p, dlogits=Fake((10, 9), F32)), lambda: M.router_select_bwd(z, i, p, p, dtype=torch.float16)):
        _refused(FL, call)
    M.router_select_bwd(z, i, p, p, dlogits=Fake((10, 8), BF), accumulate=True)
    assert FL.calls == ["moe_router_select_bwd"]


def test_quantisers_refuse(FL):
    x, o, one = Fake((10, 128), BF), Fake(3, I32), Fake(1, F32)
    for call in (lambda: M.fp4_quantize(x, fmt="fp4"), lambda: M.fp4_quantize(Fake((10, 100), BF)), lambda: M.fp4_quantize(Fake((10, 128), F32)),
                 lambda: M.fp4_quantize(x, fmt="mxfp4", scale=one), lambda: M.fp4_quantize(x, scale=Fake(2, F32)), lambda: M.fp4_quantize(x, Fake(1, I32)),
                 lambda: M.fp4_quantize(x, o, out=_pair(10, 128, 1)), lambda: M.fp4_quantize(x, out=_pair(9, 128)), lambda: M.fp4_quantize(x, out=Fake((10, 64), U8)),
                 lambda: M.fp4_quantize(x, out=(Fake((10, 64), U8, contiguous=False), _pair(10, 128)[1])),
                 lambda: M.fp4_permute(x, Fake(20, I32), 2, None), lambda: M.fp4_permute(x, Fake(20, I32), 2, o, row_of_pair=Fake(19, I32)),
                 lambda: M.fp4_quantize_weights(Fake((2, 64, 100), BF)), lambda: M.fp4_quantize_weights(Fake((2, 64, 128), BF), along="K"),
                 lambda: M.fp4_quantize_weights(Fake((2, 64, 128), BF), scale=one), lambda: M.fp4_quantize_weights(Fake((128,), BF)),
                 lambda: M.fp4_dequantize(_pair(10, 128)[0]), lambda: M.fp4_dequantize(_pair(10, 128), o), lambda: M.fp4_dequantize(_pair(10, 128), dtype=torch.float16),
                 lambda: M.fp4_dequantize(_pair(256, 128, 2, lead=2), o), lambda: M.fp4_dequantize(_pair(256, 128, 2, lead=2), scale=one)):
        _refused(FL, call)
    M.fp4_quantize(x, o, scale=one)
    M.fp4_dequantize(_pair(10, 128, 2), o, scale=one, dtype=F32)
    M.fp4_dequantize(_pair(256, 128, 2, lead=2), scale=Fake(2, F32))
    M.fp4_quantize_weights(Fake((2, 64, 128), BF), along="cols", scale=Fake(2, F32), out=_pair(128, 128, 2, lead=2))
    assert FL.calls == ["moe_fp4_quantize", "moe_fp4_dequantize", "moe_fp4_dequantize", "moe_fp4_quantize_weights"]


def test_linear_refuses(FL):
    a, w, o = _pair(10, 128, 2), _pair(512, 128, 2, lead=2), Fake(3, I32)
    for kw in (dict(act="tanh"), dict(fmt="fp4"), dict(a_scale=Fake(2, F32)), dict(w_scale=Fake(1, F32)), dict(bias=Fake((1, 256), BF)), dict(bias=Fake((2, 256), F32)),
               dict(residual=Fake((10, 128), BF)), dict(z=Fake((10, 128), BF)), dict(out=Fake((10, 256), torch.float16)), dict(out=Fake((9, 256), F32)),
               dict(out_dtype=torch.float16), dict(out_scale=Fake(1, F32)), dict(out_dtype="fp4", out=_pair(10, 128, 2)), dict(out_dtype="fp4", out_scale=Fake(2, F32))):
        _refused(FL, lambda: M.fp4_linear(a, o, w, **kw))
    _refused(FL, lambda: M.fp4_linear(a, None, w))
    _refused(FL, lambda: M.fp4_linear(_pair(10, 128, 1), o, w))              # scales of another number of experts
    _refused(FL, lambda: M.fp4_linear(_pair(10, 192, 2), o, w))
    _refused(FL, lambda: M.fp4_linear(a, o, w, fmt="mxfp4"))                  # other scales
    _refused(FL, lambda: M.fp4_linear(a[0], o, w))
    M.fp4_linear(a, o, w, act="swiglu", out_dtype="fp4", w_scale=Fake(2, F32))
    M.fp4_linear(a, o, w, out=_pair(10, 256, 2), bias=Fake((2, 256), BF), residual=Fake((10, 256), BF))
    assert FL.calls == ["moe_fp4_linear"] * 2


def test_linear_bwd_refuses(FL):
    wt, o = _pair(256, 256, 2, lead=2), Fake(3, I32)                          # K = 128, N = 256
    ok = dict(dout=Fake((10, 256), BF), a=Fake((10, 128), BF), offsets=o, wt=wt)
    for kw in (dict(dout=Fake((10, 128), BF)), dict(a=Fake((10, 64), BF)), dict(offsets=None), dict(act="relu"), dict(act="swiglu", z=Fake((10, 256), BF)),
               dict(b_layout="kk"), dict(w_scale=Fake(1, F32)), dict(fmt="mxfp4"), dict(dB=Fake((2, 256, 128), BF)), dict(b_layout="nk", dB=Fake((2, 128, 256), BF)),
               dict(da=Fake((10, 128), F32)), dict(dbias=Fake((2, 128), F32)), dict(accumulate_dw=True), dict(workspace=Fake(1 << 20, U8, is_cuda=False))):
        _refused(FL, lambda: M.fp4_linear_bwd(**{**ok, **kw}))
    M.fp4_linear_bwd(**ok, dB=Fake((2, 128, 256), BF), accumulate_dw=True)
    M.fp4_linear_bwd(**{**ok, "dout": Fake((10, 128), BF)}, act="swiglu", z=Fake((10, 256), BF), bias=True)
    assert FL.calls == ["moe_fp4_linear_bwd"] * 2
