"""What the tensor scale of the experts' rows refuses, on the host (no GPU
needed)."""
import ctypes

import pytest

import dropless_grouped_gemm_gb300 as M
from dropless_grouped_gemm_gb300 import build as B
from test_binding_checks import BF, F32, I32, U8, Fake, Lib, _refused

NULL, ALIGN, SIZE = -1, -2, -3
vp = ctypes.c_void_p
P = vp(16)          # an aligned address that nothing reads


@pytest.fixture(scope="module")
def L():
    B.build()
    return M.lib()


@pytest.mark.parametrize("kw,rc", [
    (dict(E=0), SIZE), (dict(E=1025), SIZE), (dict(rows=-1), SIZE), (dict(K=0), SIZE), (dict(K=96), SIZE), (dict(K=(1 << 23) + 64), SIZE),
    (dict(src=None), NULL), (dict(off=None), NULL), (dict(t=None), NULL), (dict(err=None), NULL), (dict(src=vp(8)), ALIGN), (dict(t=vp(18)), ALIGN)])
def test_tensor_scale_rows(L, kw, rc):
    a = dict(src=P, off=P, E=2, rows=8, K=64, t=P, err=P)
    a.update(kw)
    assert L.moe_fp4_tensor_scale_rows(a["src"], a["off"], a["E"], a["rows"], a["K"], a["t"], a["err"], None) == rc


def test_the_binding_refuses(monkeypatch):
    lib = Lib()
    monkeypatch.setattr(M, "lib", lambda: lib)
    monkeypatch.setattr(M, "_stream", lambda s=None: 0)
    monkeypatch.setattr(M, "_err_word", lambda err, dev, stream=None: err or Fake(1, I32))
    monkeypatch.setattr(M, "_empty", lambda shape, dtype, dev, stream=None: Fake(shape, dtype))
    x, o = Fake((10, 128), BF), Fake(3, I32)
    for call in (lambda: M.fp4_tensor_scale(x, per_expert=True, offsets=o), lambda: M.fp4_tensor_scale(Fake((2, 5, 128), BF), offsets=o),
                 lambda: M.fp4_tensor_scale(Fake((10, 100), BF), offsets=o), lambda: M.fp4_tensor_scale(x, offsets=Fake(1, I32)),
                 lambda: M.fp4_tensor_scale(x, offsets=Fake(3, F32)), lambda: M.fp4_tensor_scale(x, offsets=o, t=Fake(2, F32)),
                 lambda: M.fp4_tensor_scale(x, offsets=Fake(3, I32, is_cuda=False)), lambda: M.fp4_tensor_scale(Fake((10, 128), U8), offsets=o)):
        _refused(lib, call)
    M.fp4_tensor_scale(x, offsets=o)
    M.fp4_tensor_scale(x)
    assert lib.calls == ["moe_fp4_tensor_scale_rows", "moe_fp4_tensor_scale"]
