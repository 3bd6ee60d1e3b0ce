"""What the operators around the expert MLP refuse, on the host and before
anything is enqueued: the C entry points' return codes, and the binding's
checks (no GPU needed)."""
import ctypes

import pytest
import torch

import dropless_grouped_gemm_gb300 as M
from dropless_grouped_gemm_gb300 import build as B

NULL, ALIGN, SIZE, ARG, WS = -1, -2, -3, -4, -6
vp = ctypes.c_void_p
P = vp(16)          # an aligned address that nothing reads


@pytest.fixture(scope="module")
def L():
    B.build()
    return M.lib()


def _loss(L, **kw):
    a = dict(logits=P, lt=0, idx=P, T=4, E=8, k=2, seg=None, S=1, mask=None, loss=P, counts=P, lse=P,
             n_valid=P, ws=P, wsb=1 << 20, err=P)
    a.update(kw)
    return L.moe_router_loss(a["logits"], a["lt"], a["idx"], a["T"], a["E"], a["k"], a["seg"], a["S"],
                             a["mask"], a["loss"], a["counts"], a["lse"], a["n_valid"], a["ws"],
                             a["wsb"], a["err"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), SIZE), (dict(E=0), SIZE), (dict(E=1025), SIZE), (dict(k=0), SIZE), (dict(k=9), SIZE),
    (dict(S=0), SIZE), (dict(S=4097, seg=P), SIZE), (dict(S=2), SIZE),        # S > 1 needs offsets
    (dict(T=(1 << 30) + 1), SIZE), (dict(T=1 << 29, k=8), SIZE), (dict(lt=2), ARG),
    (dict(logits=None), NULL), (dict(idx=None), NULL), (dict(loss=None), NULL), (dict(counts=None), NULL),
    (dict(lse=None), NULL), (dict(n_valid=None), NULL), (dict(err=None), NULL), (dict(ws=None), NULL),
    (dict(logits=vp(20)), ALIGN), (dict(ws=vp(8)), ALIGN), (dict(wsb=64), WS)])
def test_router_loss(L, kw, rc):
    assert _loss(L, **kw) == rc


def _loss_bwd(L, **kw):
    a = dict(logits=P, lt=0, idx=P, T=4, E=8, k=2, seg=None, S=1, lse=P, counts=P, n_valid=P, dloss=P,
             probs=P, dprobs=P, out=P, ot=0)
    a.update(kw)
    return L.moe_router_loss_bwd(a["logits"], a["lt"], a["idx"], a["T"], a["E"], a["k"], a["seg"], a["S"],
                                 None, a["lse"], a["counts"], a["n_valid"], a["dloss"], a["probs"],
                                 a["dprobs"], a["out"], a["ot"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(E=0), SIZE), (dict(k=9), SIZE), (dict(S=3), SIZE), (dict(lt=7), ARG), (dict(ot=-1), ARG),
    (dict(probs=None), NULL), (dict(dprobs=None), NULL), (dict(dloss=None), NULL), (dict(out=None), NULL),
    (dict(lse=None), NULL), (dict(counts=None), NULL), (dict(out=vp(24)), ALIGN), (dict(T=0), 0)])
def test_router_loss_bwd(L, kw, rc):
    assert _loss_bwd(L, **kw) == rc


def test_workspace_sizes(L):
    assert L.moe_router_loss_workspace_size(-1, 8, 1) == 0
    assert L.moe_router_loss_workspace_size(4, 8, 0) == 0
    assert L.moe_router_loss_workspace_size(0, 8, 1) > 0
    # at least a row of sums and one of counts per sequence, and below the logits
    assert 2 * 256 * 4 * 16 < L.moe_router_loss_workspace_size(65536, 256, 16) < 65536 * 256 * 4
    assert L.moe_grouped_linear_bwd_workspace_size(0, 8, 64) == 0
    assert L.moe_grouped_linear_bwd_workspace_size(4, 1000, 64) >= 8 * 64 * 4


def _linear(L, **kw):
    a = dict(a=P, off=P, E=2, M=8, K=64, N=128, B=P, lay=0, bias=P, act=3, res=P, z=P, out=P, ot=1, err=P)
    a.update(kw)
    return L.moe_grouped_linear(a["a"], a["off"], a["E"], a["M"], a["K"], a["N"], a["B"], a["lay"], a["bias"],
                                a["act"], a["res"], a["z"], a["out"], a["ot"], a["err"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(E=0), SIZE), (dict(E=1025), SIZE), (dict(M=-1), SIZE), (dict(K=96), SIZE), (dict(N=32), SIZE),
    (dict(K=0), SIZE), (dict(N=(1 << 23) + 64), SIZE), (dict(off=None), SIZE),      # two experts need offsets
    (dict(lay=2), ARG), (dict(act=7), ARG), (dict(act=-1), ARG), (dict(ot=2), ARG),
    (dict(a=None), NULL), (dict(B=None), NULL), (dict(out=None), NULL), (dict(err=None), NULL),
    (dict(a=vp(8)), ALIGN), (dict(bias=vp(8)), ALIGN), (dict(res=vp(8)), ALIGN), (dict(z=vp(8)), ALIGN),
    (dict(out=vp(8)), ALIGN), (dict(M=0), 0)])
def test_linear(L, kw, rc):
    assert _linear(L, **kw) == rc


def _linear_bwd(L, **kw):
    a = dict(dout=P, z=P, a=P, off=P, E=2, M=8, K=64, N=128, B=P, lay=0, act=0, fl=0, dz=P, da=P, dB=P, db=P,
             ws=P, wsb=1 << 20, err=P)
    a.update(kw)
    return L.moe_grouped_linear_bwd(a["dout"], a["z"], a["a"], a["off"], a["E"], a["M"], a["K"], a["N"], a["B"],
                                    a["lay"], a["act"], a["fl"], a["dz"], a["da"], a["dB"], a["db"], a["ws"],
                                    a["wsb"], a["err"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(K=32), SIZE), (dict(off=None), SIZE), (dict(act=9), ARG), (dict(lay=-1), ARG), (dict(fl=1), ARG),
    (dict(dout=None), NULL), (dict(z=None), NULL), (dict(dz=None), NULL), (dict(a=None), NULL),
    (dict(B=None), NULL), (dict(err=None), NULL), (dict(ws=None), NULL), (dict(ws=vp(4)), ALIGN),
    (dict(wsb=16), WS), (dict(da=vp(8)), ALIGN), (dict(db=vp(8)), ALIGN), (dict(z=vp(8)), ALIGN)])
def test_linear_bwd(L, kw, rc):
    assert _linear_bwd(L, **kw) == rc


def test_checkpoints(L):
    assert L.moe_checkpoint_pack(P, 4, 96, P, P, None) == SIZE
    assert L.moe_checkpoint_pack(P, -1, 64, P, P, None) == SIZE
    assert L.moe_checkpoint_pack(None, 4, 64, P, P, None) == NULL
    assert L.moe_checkpoint_pack(vp(8), 4, 64, P, P, None) == ALIGN
    assert L.moe_checkpoint_pack(None, 0, 64, None, None, None) == 0
    assert L.moe_checkpoint_unpack(P, P, 4, 100, P, None) == SIZE
    assert L.moe_checkpoint_unpack(P, None, 4, 64, P, None) == NULL
    assert L.moe_checkpoint_unpack(P, P, 4, 64, vp(8), None) == ALIGN
    assert L.moe_permute_checkpoint(P, P, None, P, 4, 0, 64, 4, P, None) == SIZE
    assert L.moe_permute_checkpoint(P, P, None, None, 4, 1, 64, 4, P, None) == NULL
    assert L.moe_permute_checkpoint(None, P, None, P, 4, 1, 64, 4, P, None) == NULL
    assert L.moe_permute_checkpoint(vp(4), P, None, P, 4, 1, 64, 4, P, None) == ALIGN
    assert L.moe_permute_checkpoint(None, None, None, None, 4, 1, 64, 0, None, None) == 0
    f = L.moe_grouped_mlp_fwd_ckpt
    assert f(P, P, 2, 8, 96, 64, P, P, 0, P, P, P, P, P, None) == SIZE
    assert f(P, P, 2, 8, 64, 64, P, P, 3, P, P, P, P, P, None) == ARG        # MLP activations only
    assert f(P, P, 2, 8, 64, 64, P, P, 0, None, P, P, P, P, None) == NULL
    assert f(P, P, 2, 8, 64, 64, P, P, 0, P, vp(2), P, P, P, None) == ALIGN
    assert f(P, P, 2, 0, 64, 64, P, P, 0, None, None, None, None, P, None) == 0
    b = L.moe_grouped_mlp_bwd_routed_ckpt
    ok = [P, P, P, P, P, P, P, 2, 8, 64, 64, P, P, 0, 0, P, P, P, P, P, P, P, None]
    for i, v, rc in ((7, 0, SIZE), (9, 32, SIZE), (13, 4, ARG), (14, 1, ARG), (1, None, NULL), (2, None, NULL),
                     (5, None, NULL), (1, vp(8), ALIGN), (2, vp(2), ALIGN)):
        a = list(ok)
        a[i] = v
        assert b(*a) == rc, (i, v)


def test_binding_refusals():
    z, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(M.MoeError, match="CUDA"):
        M.router_loss(z, i)
    with pytest.raises(M.MoeError, match="float32 or torch.bfloat16"):
        M.router_loss(z.half(), i)
    a, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(1, 64, 64, dtype=torch.bfloat16)
    with pytest.raises(M.MoeError, match="CUDA"):
        M.grouped_linear(a, None, w)
    with pytest.raises(M.MoeError, match="CUDA"):
        M.checkpoint_pack(a)
    with pytest.raises(M.MoeError, match="CUDA"):
        M.checkpoint_unpack(a.view(torch.uint8), a.view(torch.uint8))


@pytest.mark.gpu
def test_binding_refusals_on_the_gpu():
    dev = "cuda"
    a = torch.zeros(4, 64, dtype=torch.bfloat16, device=dev)
    w = torch.zeros(2, 64, 128, dtype=torch.bfloat16, device=dev)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=dev)
    bad = [
        lambda: M.grouped_linear(a, off, w, "tanh"),
        lambda: M.grouped_linear(a, off, w, b_layout="kk"),
        lambda: M.grouped_linear(a, off[:2], w),
        lambda: M.grouped_linear(a, None, w),                                  # two experts, no offsets
        lambda: M.grouped_linear(a, off, w, bias=a[0]),
        lambda: M.grouped_linear(a, off, w, residual=a),
        lambda: M.grouped_linear(a, off, w, out_dtype=torch.float16),
        lambda: M.grouped_linear(a[:, ::2], off, w),
        lambda: M.grouped_linear_bwd(a, a, off, w),                            # dout has N columns
        lambda: M.grouped_linear_bwd(a, a, off, w, "swiglu"),                  # no z
        lambda: M.router_loss(a, off[None, :2]),                               # one token against four
        lambda: M.checkpoint_pack(torch.zeros(4, 96, dtype=torch.bfloat16, device=dev)),
        lambda: M.checkpoint_unpack(torch.zeros(4, 64, dtype=torch.uint8, device=dev),
                                    torch.zeros(4, 3, dtype=torch.uint8, device=dev)),
        lambda: M.permute_checkpoint(torch.zeros(4, 64, dtype=torch.uint8, device=dev),
                                     torch.zeros(4, 2, dtype=torch.uint8, device=dev), off, 2,
                                     row_of_pair=off),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(M.MoeError):
            f()
            pytest.fail(f"case {i} was accepted")
    with pytest.raises(ValueError):
        M.grouped_linear_bwd(torch.zeros(4, 128, dtype=torch.bfloat16, device=dev), a, off, w,
                             accumulate_dw=True)
