"""Calls given a stream of their own: their error words, workspaces and
outputs belong to it."""
import numpy as np
import pytest
import torch

import workloads as W
from _helpers import cuda_i32

pytestmark = pytest.mark.gpu


def _busy():
    """Some 10 ms of ordinary work on the current stream."""
    x = torch.empty(1 << 28, device="cuda")
    for _ in range(40):
        x.fill_(1.0)
    return x


def _old_calls(M):
    """Entry points with a device error word, each on inputs that set it (or
    0: sets nothing), as functions of the stream."""
    idx = cuda_i32(np.full((64, 2), 99))
    z = torch.zeros((8, 16), device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, W1, W2 = torch.zeros((64, 128), **bf), torch.zeros((2, 128, 256), **bf), torch.zeros((2, 128, 128), **bf)
    h, a = torch.zeros((64, 256), **bf), torch.zeros((64, 128), **bf)
    bad, odd = cuda_i32([0, 64, 32]), cuda_i32([0, 33, 64])
    por = cuda_i32(np.arange(64))
    probs = torch.ones((64, 1), device="cuda")
    O = M.DEV_BAD_OFFSETS
    return {
        "route_offsets": (lambda s: M.route_offsets(idx, 4, stream=s)["err"], M.DEV_BAD_EXPERT),
        "route_logits": (lambda s: M.route_logits(z, 4, M_cap=4, stream=s)["err"], M.DEV_OVERFLOW),
        "grouped_mlp_fwd": (lambda s: M.grouped_mlp_fwd(x, bad, W1, W2, stream=s)[-1], O),
        "grouped_mlp_fwd_gather": (lambda s: M.grouped_mlp_fwd_gather(x, por, 1, bad, W1, W2, stream=s)[-1], O),
        "grouped_mlp_bwd": (lambda s: M.grouped_mlp_bwd(x, h, a, x, bad, W1, W2, stream=s)[-1], O),
        "grouped_mlp_bwd_routed": (lambda s: M.grouped_mlp_bwd_routed(x, h, x, por, probs, bad, W1, W2, stream=s)[-1], O),
        "grouped_mlp_bwd_routed_gather": (lambda s: M.grouped_mlp_bwd_routed_gather(x, x, por, 1, h, probs, bad, W1, W2, stream=s)[-1], O),
        "grouped_gemm": (lambda s: M.grouped_gemm(a, bad, W2, stream=s)[-1], O),
        "mx_quantize": (lambda s: M.mx_quantize(x, odd, stream=s)[-1], O),
        "mx_quantize_tiled": (lambda s: M.mx_quantize_tiled(x, odd, stream=s)[-1], O),
    }


@pytest.mark.parametrize("name", ["route_offsets", "route_logits", "grouped_mlp_fwd", "grouped_mlp_fwd_gather",
                                  "grouped_mlp_bwd", "grouped_mlp_bwd_routed", "grouped_mlp_bwd_routed_gather",
                                  "grouped_gemm", "mx_quantize", "mx_quantize_tiled"])
def test_error_words_follow_the_stream(name):
    """The current stream is busy, so what it zeroes is zeroed late: a word
    zeroed there after the side stream's kernel has set it would read 0."""
    import dropless_grouped_gemm_gb300 as M
    call, bits = _old_calls(M)[name]
    st = torch.cuda.Stream()
    want = call(None)
    torch.cuda.synchronize()
    assert int(want.item()) == bits
    M._ERR_WORDS.clear()
    keep = _busy()
    got = call(st)
    torch.cuda.synchronize()
    del keep
    assert int(got.item()) == bits


def test_error_words_made_in_inference_mode():
    """A word handed out later is an ordinary tensor, whatever mode the call
    that made its 64 ran in."""
    import dropless_grouped_gemm_gb300 as M
    a = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda")
    B = torch.ones((64, 64), dtype=torch.bfloat16, device="cuda")
    M._ERR_WORDS.clear()
    with torch.inference_mode():
        _, _, e0 = M.grouped_linear(a, None, B)
        e0.zero_()
    _, _, e1 = M.grouped_linear(a, None, B)
    e1.zero_()
    assert not e1.is_inference() and int(e0.item()) == 0 and int(e1.item()) == 0


def _linear_case():
    E, M, K, N = 3, 400, 128, 256
    off = cuda_i32([0, 100, 250, 400])
    a = W.normal((M, K), (40, W.X, 0), 1.0, "cuda")
    B = W.normal((E, K, N), (40, W.W2, 1), 0.05, "cuda")
    z = W.normal((M, N), (40, W.X, 5), 1.5, "cuda")
    dout = W.normal((M, N), (40, W.DO, 0), 1.0, "cuda")
    return E, M, K, N, off, a, B, z, dout


def test_outputs_do_not_come_from_memory_the_current_stream_still_writes():
    import dropless_grouped_gemm_gb300 as M_
    E, M, K, N, off, a, B, z, dout = _linear_case()
    want = M_.grouped_linear_bwd(dout, a, off, B, "silu", z, True)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    keep = _busy()
    # blocks of the outputs' sizes, freed with a write to each still queued
    old = [torch.empty_like(t) for t in want[:4]]
    for t in old:
        t.fill_(float("nan"))
    del t, old
    got = M_.grouped_linear_bwd(dout, a, off, B, "silu", z, True, stream=st)
    torch.cuda.synchronize()
    del keep
    for x, y in zip(got[:4], want[:4]):
        assert torch.equal(x, y)


def test_outputs_are_not_reused_while_the_current_stream_reads_them():
    import dropless_grouped_gemm_gb300 as M_
    E, M, K, N, off, a, B, z, dout = _linear_case()
    want = M_.grouped_linear_bwd(dout, a, off, B, "silu", z, True)
    other = W.normal((M, N), (41, W.DO, 0), 1.0, "cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = M_.grouped_linear_bwd(dout, a, off, B, "silu", z, True, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    keep = _busy()
    copies = [t.clone() for t in got[:4]]                 # queued behind the busy work
    del got
    again = M_.grouped_linear_bwd(other, a, off, B, "silu", z, True, stream=st)
    torch.cuda.synchronize()
    del keep, again
    for x, y in zip(copies, want[:4]):
        assert torch.equal(x, y)


def _pointer(M_, name, index, monkeypatch):
    """The argument `index` of every call of the C entry `name`."""
    seen, f = [], getattr(M_.lib(), name)

    def spy(*args):
        seen.append(args[index])
        return f(*args)
    monkeypatch.setattr(M_.lib(), name, spy)
    return seen


def test_workspaces_do_not_come_from_memory_the_current_stream_still_uses(monkeypatch):
    import dropless_grouped_gemm_gb300 as M_
    E, M, K, N, off, a, B, z, dout = _linear_case()
    lin = _pointer(M_, "moe_grouped_linear_bwd", 16, monkeypatch)
    loss = _pointer(M_, "moe_router_loss", 13, monkeypatch)
    route = _pointer(M_, "moe_route_offsets", 11, monkeypatch)
    logits = torch.randn((300, 64), device="cuda")
    idx = logits.topk(2).indices.int()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()

    def calls(s):
        M_.grouped_linear_bwd(dout, a, off, B, "silu", z, True, stream=s)
        M_.router_loss(logits, idx, stream=s)
        M_.route_offsets(idx, 64, stream=s)
    keep = _busy()
    calls(None)                                           # their scratch is freed on return
    calls(st)
    torch.cuda.synchronize()
    del keep
    for p in (lin, loss, route):
        assert len(p) == 2 and p[0] != p[1], p


def test_workspaces_are_not_reused_while_the_call_is_still_queued():
    """The side stream is busy, so its call runs late; tensors of the
    workspace's size are made and filled on the current stream meanwhile."""
    import dropless_grouped_gemm_gb300 as M_
    E, M, K, N, off, a, B, z, dout = _linear_case()
    want = M_.grouped_linear_bwd(dout, a, off, B, "silu", z, True)
    size = M_.grouped_linear_bwd_workspace_size(E, M, N)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        keep = _busy()
    got = M_.grouped_linear_bwd(dout, a, off, B, "silu", z, True, stream=st)
    junk = [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(16)]
    torch.cuda.synchronize()
    del keep, junk
    for x, y in zip(got[:4], want[:4]):
        assert torch.equal(x, y)


def test_a_call_on_a_forked_stream_captures():
    """Everything that the call makes lies in the graph's memory, the zeroing
    of its error word in the graph."""
    import dropless_grouped_gemm_gb300 as M_
    E, M, K, N, off, a, B, z, dout = _linear_case()
    want = M_.grouped_linear_bwd(dout, a, off, B, "silu", z, True)
    bad = cuda_i32([0, 400, 100, 400])
    torch.cuda.synchronize()
    main, side, g = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        side.wait_stream(main)
        got = M_.grouped_linear_bwd(dout, a, off, B, "silu", z, True, stream=side)
        _, _, err = M_.grouped_linear(a, bad, B, stream=side)
        main.wait_stream(side)
    for _ in range(2):
        for t in got[:4]:
            t.zero_()
        err.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert int(got[4].item()) == 0 and int(err.item()) == M_.DEV_BAD_OFFSETS
        for x, y in zip(got[:4], want[:4]):
            assert torch.equal(x, y)
