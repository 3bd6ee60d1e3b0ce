"""The MoE block example: gate, router losses, experts with H in 8 bits and a
shared expert, run together.  Its gradients against a float64 composition of
the oracle's operators (on the same routing and the same 8-bit checkpoints),
and a few training steps."""
import os
import sys

import numpy as np
import pytest
import torch

import oracle as O
from _helpers import assert_rms_close, f64

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_gradients():
    import moe_block as B
    T, d, E, k, n, ns = 300, 128, 64, 3, 64, 192
    w = {name: t.to(torch.bfloat16) for name, t in B.init(E, d, n, ns, 3).items()}
    w["bg"] = torch.linspace(-1, 1, E, device="cuda").to(torch.bfloat16)
    x = torch.randn((T, d), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    seg = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    mask = torch.ones(T, dtype=torch.uint8, device="cuda")
    mask[250:] = 0
    out, losses, saved = B.forward(x, w, k, seg, mask)
    dout = torch.randn((T, d), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(torch.bfloat16)
    dl = torch.tensor([0.5, 0.1], device="cuda")
    grads = B.backward(dout, dl, saved, w)
    torch.cuda.synchronize()
    assert int(saved["err"].item()) == 0
    W = {name: f64(t) for name, t in w.items()}
    r = saved["r"]
    idx, probs = r["topk_idx"].cpu().numpy(), r["probs"].cpu().numpy().astype(np.float64)
    # forward
    logits = f64(x) @ W["Wg"] + W["bg"]
    assert np.abs(saved["logits"].cpu().numpy() - logits).max() <= 2.0 ** -16 * np.abs(logits).max()
    ro = O.route_offsets(idx, E, 1)
    off, por = ro["offsets"], ro["pair_of_row"]
    ref = O.router_loss(saved["logits"].cpu().numpy(), idx, seg.tolist(), mask.cpu().numpy())
    assert np.abs(losses.cpu().numpy() - ref["loss"]).max() <= 1e-5 * ref["loss"].max()
    _, _, Y = O.grouped_mlp_fwd(O.permute(f64(x), por, k), off, W["W1"], W["W2"], "swiglu")
    routed = O.unpermute(Y, ro["row_of_pair"], T, k, probs)
    s = f64(saved["s"])
    assert_rms_close(s, O.linear_act(f64(x) @ W["Ws1"], "swiglu"), "block shared activation")
    assert_rms_close(f64(out), s @ W["Ws2"] + routed, "block output")
    # backward, on what the forward kept
    x8 = O.checkpoint_unpack(*O.checkpoint_pack(f64(x)))
    g = f64(dout)
    ds = O.bf16_round(g @ W["Ws2"].T)
    dz = O.bf16_round(O.linear_dact(f64(saved["z"]), ds, "swiglu"))
    h8 = O.checkpoint_unpack(saved["h_q"].cpu().numpy(), saved["h_s"].cpu().numpy())
    x8p, dop = O.permute(x8, por, k), O.permute(g, por, k)
    _, dXp, dW1, dW2, _, dS = O.grouped_mlp_bwd_routed(x8p, h8, dop, probs.reshape(-1)[por], off,
                                                       W["W1"], W["W2"], "swiglu", round_out=False)
    dprobs = np.zeros((T, k))
    dprobs.reshape(-1)[por] = dS
    dlog = O.bf16_round(O.router_loss_bwd(saved["logits"].cpu().numpy(), idx, f64(dl), probs, dprobs,
                                          seg.tolist(), mask.cpu().numpy()))
    dx = dz @ W["Ws1"].T + O.unpermute(dXp, ro["row_of_pair"], T, k) + dlog @ W["Wg"].T
    for name, want in (("Ws2", s.T @ g), ("Ws1", x8.T @ dz), ("W1", dW1), ("W2", dW2),
                       ("Wg", x8.T @ dlog), ("x", dx)):
        assert_rms_close(f64(grads[name]), want, f"block d{name}")
    assert_rms_close(f64(grads["bg"]), dlog.sum(axis=0), "block dbg")


def test_training_steps_lower_both_losses():
    import moe_block as B
    h = B.train(steps=12, T=512, balance=0.1)
    assert np.isfinite(np.array(h)).all()
    assert h[-1][0] < 0.9 * h[0][0]        # the regression
    assert h[-1][1] < h[0][1]              # the balance of the uneven router
