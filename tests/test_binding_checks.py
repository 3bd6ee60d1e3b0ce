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


def _ckpt_fwd(**kw):
    a = dict(x_perm=Fake((96, 128), BF), offsets=Fake(3, I32), W1=Fake((2, 128, 256), BF),
             W2=Fake((2, 128, 128), BF), h_q=Fake((96, 256), U8), h_s=Fake((96, 8), U8),
             a=Fake((96, 128), BF), y_perm=Fake((96, 128), BF))
    a.update(kw)
    return M.grouped_mlp_fwd_ckpt(**a)


@pytest.mark.parametrize("bad", [
    dict(a=Fake((95, 128), BF)), dict(a=Fake((96, 128), F32)), dict(y_perm=Fake((96, 64), BF)),
    dict(y_perm=Fake((96, 128), BF, is_cuda=False)), dict(y_perm=Fake((96, 128), BF, contiguous=False)),
    dict(h_q=Fake((96, 128), U8)), dict(h_s=Fake((96, 4), U8)), dict(act="relu")])
def test_mlp_fwd_ckpt_refuses_buffers_that_do_not_fit(L, bad):
    _refused(L, lambda: _ckpt_fwd(**bad))


def _ckpt_bwd(**kw):
    a = dict(x_perm=Fake((96, 128), BF), h_q=Fake((96, 256), U8), h_s=Fake((96, 8), U8),
             do_perm=Fake((96, 128), BF), pair_of_row=Fake(96, I32), probs=Fake((50, 2), F32),
             offsets=Fake(3, I32), W1=Fake((2, 128, 256), BF), W2=Fake((2, 128, 128), BF),
             dh=Fake((96, 256), BF), a_scaled=Fake((96, 128), BF), ds_part=Fake((96, 1), F32),
             dx_perm=Fake((96, 128), BF), dW1=Fake((2, 128, 256), BF), dW2=Fake((2, 128, 128), BF))
    a.update(kw)
    return M.grouped_mlp_bwd_routed_ckpt(**a)


@pytest.mark.parametrize("bad", [
    dict(do_perm=Fake((95, 128), BF)), dict(pair_of_row=Fake(95, I32)), dict(offsets=Fake(4, I32)),
    dict(W1=Fake((2, 128, 128), BF)), dict(W2=Fake((2, 128, 64), BF)), dict(dh=Fake((96, 128), BF)),
    dict(dh=Fake((96, 256), F32)), dict(a_scaled=Fake((90, 128), BF)), dict(ds_part=Fake((96, 2), F32)),
    dict(ds_part=Fake((96, 1), BF)), dict(dx_perm=Fake((96, 64), BF)), dict(dW1=Fake((1, 128, 256), BF)),
    dict(dW2=Fake((2, 128, 128), BF, is_cuda=False)), dict(dW2=Fake((2, 128, 128), BF, contiguous=False)),
    dict(h_q=Fake((90, 256), U8)), dict(act="none")])
def test_mlp_bwd_ckpt_refuses_buffers_that_do_not_fit(L, bad):
    _refused(L, lambda: _ckpt_bwd(**bad))


def test_mlp_ckpt_calls_take_buffers_that_fit(L):
    _ckpt_fwd()
    _ckpt_fwd(act="srelu", W1=Fake((2, 128, 128), BF), h_q=Fake((96, 128), U8), h_s=Fake((96, 4), U8))
    _ckpt_fwd(h_q=None, h_s=None, a=None, y_perm=None)
    _ckpt_bwd()
    _ckpt_bwd(dh=None, a_scaled=None, ds_part=None, dx_perm=None, dW1=None, dW2=None)
    assert L.calls == ["moe_grouped_mlp_fwd_ckpt"] * 3 + ["moe_grouped_mlp_bwd_routed_ckpt"] * 2


@pytest.mark.parametrize("ws", [Fake(1 << 20, U8, is_cuda=False), Fake(1 << 20, U8, contiguous=False)])
def test_workspaces_must_be_contiguous_cuda_memory(L, ws):
    z, i = Fake((10, 8), F32), Fake((10, 2), I32)
    _refused(L, lambda: M.router_loss(z, i, workspace=ws))
    _refused(L, lambda: M.route_offsets(i, 8, workspace=ws))
    _refused(L, lambda: M.route_logits(z, 2, workspace=ws))
    x = Fake((10, 64), BF)
    _refused(L, lambda: M.grouped_linear_bwd(x, x, None, Fake((64, 64), BF), bias=True, workspace=ws))


def test_workspaces_of_any_type(L):
    z, i, x = Fake((10, 8), F32), Fake((10, 2), I32), Fake((10, 64), BF)
    M.router_loss(z, i, workspace=Fake(4096, F32))
    M.grouped_linear_bwd(x, x, None, Fake((64, 64), BF), bias=True, workspace=Fake(4096, I32))
    assert L.calls == ["moe_router_loss", "moe_grouped_linear_bwd"]
