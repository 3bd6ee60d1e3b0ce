"""What the binding checks of the tensors it is given, on the CPU: stand-ins
for CUDA tensors and for the library, which no refused call may reach."""
import pytest
import torch

import dropless_grouped_gemm_gb300 as M

F32, BF, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


class Fake:
    """As much of a tensor as the binding asks about."""

    def __init__(self, shape, dtype, is_cuda=True, contiguous=True):
        self.shape = tuple(shape) if isinstance(shape, (tuple, list, torch.Size)) else (shape,)
        self.dtype, self.is_cuda, self._contiguous = dtype, is_cuda, contiguous
        self.device = torch.device("cuda", 0)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def dim(self):
        return len(self.shape)

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return self._contiguous

    def data_ptr(self):
        return 16


class Lib:
    """Counts the calls of the library; sizes are 1024 bytes."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def f(*args):
            if name.endswith("_workspace_size"):
                return 1024
            self.calls.append(name)
            return 0
        return f


@pytest.fixture
def L(monkeypatch):
    lib = Lib()
    monkeypatch.setattr(M, "lib", lambda: lib)
    monkeypatch.setattr(M, "_stream", lambda s=None: 0)
    monkeypatch.setattr(M, "_err_word", lambda err, dev, stream=None: err or Fake(1, I32))
    monkeypatch.setattr(M, "_empty", lambda shape, dtype, dev, stream=None: Fake(shape, dtype))
    monkeypatch.setattr(M, "_scratch", lambda n, dev, stream=None: Fake(n, U8))
    return lib


def _refused(L, call):
    with pytest.raises((M.MoeError, ValueError)):
        call()
    assert not L.calls


def _loss_out(**kw):
    o = {"loss": Fake(2, F32), "counts": Fake((3, 8), I32), "lse": Fake(10, F32), "n_valid": Fake(3, I32)}
    o.update(kw)
    return o


def _loss(out):
    return M.router_loss(Fake((10, 8), F32), Fake((10, 2), I32), Fake(4, I32), out=out)


@pytest.mark.parametrize("bad", [
    dict(loss=Fake(1, F32)), dict(loss=Fake(2, BF)), dict(counts=Fake((2, 8), I32)),
    dict(counts=Fake((3, 8), torch.int64)), dict(counts=Fake((3, 8), I32, contiguous=False)),
    dict(lse=Fake(9, F32)), dict(lse=Fake(10, F32, is_cuda=False)), dict(n_valid=Fake(4, I32)),
    dict(n_valid=None), dict(err=Fake(1, torch.int64))])
def test_router_loss_refuses_buffers_that_do_not_fit(L, bad, monkeypatch):
    monkeypatch.setattr(M, "_err_word", lambda err, dev, stream=None: M._need(err, I32, "err") or err)
    _refused(L, lambda: _loss(_loss_out(**bad)))


def test_router_loss_takes_buffers_that_fit(L):
    o = _loss_out()
    assert _loss(o) is o and L.calls == ["moe_router_loss"]
