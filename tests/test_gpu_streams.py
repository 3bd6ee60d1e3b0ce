"""Calls given a stream of their own: their error words belong to it."""
import numpy as np
import pytest
import torch

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
