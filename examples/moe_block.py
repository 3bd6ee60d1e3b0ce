"""A trainable MoE block out of this library's calls, forward and backward.

    python examples/moe_block.py [--steps N] [--tokens T]

out = shared(x) + routed(x):

  gate      logits = x Wg + bg in float32 (grouped_linear, dense)
  router    top-k, probabilities and routing layout (route_logits); the
            load-balance and z losses with their counts (router_loss)
  experts   gated MLP over the routed rows, H kept in 8 bits
            (grouped_mlp_fwd_ckpt), combined with the probabilities (unpermute)
  shared    a dense gated MLP (grouped_linear with "swiglu"), whose second
            product adds the routed output as its residual

Between forward and backward the block keeps the token rows and H in 8 bits
(checkpoint_pack, h_q / h_s), the shared expert's pre-activation, and the
router's small tensors.  The backward gathers the expert-major rows back from
the packed tokens (permute_checkpoint), runs the routed backward from the
8-bit H, and sends the router's gradient - its losses' and the probabilities'
- through the gate (router_loss_bwd, grouped_linear_bwd).
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import dropless_grouped_gemm_gb300 as M  # noqa: E402

BF = torch.bfloat16


def init(E: int, d: int, n: int, n_shared: int, seed: int = 0, device="cuda") -> dict:
    """float32 master weights; W1 and Ws1 hold interleaved (gate, up) columns."""
    g = torch.Generator(device=device).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
    return {"Wg": r(d, E) * d ** -0.5, "bg": torch.zeros(E, device=device),
            "W1": r(E, d, 2 * n) * d ** -0.5, "W2": r(E, n, d) * n ** -0.5,
            "Ws1": r(d, 2 * n_shared) * d ** -0.5, "Ws2": r(n_shared, d) * n_shared ** -0.5}


def forward(x: torch.Tensor, w: dict, k: int, seg_offsets=None, token_mask=None):
    """x [T, d] bf16, w bf16 weights.  Returns (out bf16 [T, d], losses [2]
    float32 (balance, z), what the backward needs)."""
    T = x.shape[0]
    logits, _, err = M.grouped_linear(x, None, w["Wg"], bias=w["bg"], out_dtype=torch.float32)
    r = M.route_logits(logits, k, err=err)
    loss = M.router_loss(logits, r["topk_idx"], seg_offsets, token_mask, err=err)
    x_q, x_s = M.checkpoint_pack(x)
    x_perm = M.permute(x, r["pair_of_row"], k, row_of_pair=r["row_of_pair"])
    h_q, h_s, _, y, _ = M.grouped_mlp_fwd_ckpt(x_perm, r["offsets"], w["W1"], w["W2"], err=err)
    routed, _ = M.unpermute(y, r["row_of_pair"], T, k, probs=r["probs"])
    s, z, _ = M.grouped_linear(x, None, w["Ws1"], "swiglu", save_z=True, err=err)
    out, _, _ = M.grouped_linear(s, None, w["Ws2"], residual=routed, err=err)
    saved = {"x_q": x_q, "x_s": x_s, "logits": logits, "r": r, "loss": loss, "h_q": h_q, "h_s": h_s,
             "s": s, "z": z, "k": k, "seg": seg_offsets, "mask": token_mask, "err": err}
    return out, loss["loss"], saved


def backward(dout: torch.Tensor, dlosses: torch.Tensor, saved: dict, w: dict) -> dict:
    """Gradients of the weights and of x, from dout [T, d] bf16 and the two
    losses' gradients dlosses [2] float32."""
    T, k, r, err = dout.shape[0], saved["k"], saved["r"], saved["err"]
    x8 = M.checkpoint_unpack(saved["x_q"], saved["x_s"])
    _, ds, dWs2, _, _ = M.grouped_linear_bwd(dout, saved["s"], None, w["Ws2"], err=err)
    _, dx_shared, dWs1, _, _ = M.grouped_linear_bwd(ds, x8, None, w["Ws1"], "swiglu", z=saved["z"],
                                                    err=err)
    x_perm = M.permute_checkpoint(saved["x_q"], saved["x_s"], r["pair_of_row"], k,
                                  row_of_pair=r["row_of_pair"])
    do_perm = M.permute(dout, r["pair_of_row"], k, row_of_pair=r["row_of_pair"])
    _, _, part, dx_perm, dW1, dW2, _ = M.grouped_mlp_bwd_routed_ckpt(
        x_perm, saved["h_q"], saved["h_s"], do_perm, r["pair_of_row"], r["probs"], r["offsets"],
        w["W1"], w["W2"], err=err)
    dprobs = M.router_grad_rows(part, r["row_of_pair"], T, k)
    dx_routed, _ = M.unpermute(dx_perm, r["row_of_pair"], T, k)
    dlogits = M.router_loss_bwd(saved["logits"], r["topk_idx"], saved["loss"], dlosses, r["probs"],
                                dprobs, saved["seg"], saved["mask"], dtype=BF)
    _, dx_gate, dWg, dbg, _ = M.grouped_linear_bwd(dlogits, x8, None, w["Wg"], bias=True, err=err)
    dx = dx_shared.float() + dx_routed.float() + dx_gate.float()
    return {"Wg": dWg, "bg": dbg[0], "W1": dW1, "W2": dW2, "Ws1": dWs1, "Ws2": dWs2, "x": dx}


def train(steps: int = 20, T: int = 1024, d: int = 256, E: int = 64, k: int = 4, n: int = 128,
          n_shared: int = 256, lr: float = 0.5, balance: float = 1e-2, z: float = 1e-3, seed: int = 0):
    """A few steps of gradient descent on a random regression; returns the
    losses (mean squared error, balance, z) of each step."""
    w32 = init(E, d, n, n_shared, seed)
    w32["bg"][: E // 8] += 1.5            # a router that starts out uneven
    teacher = {name: t.to(BF) for name, t in init(E, d, n, n_shared, seed + 1).items()}
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    x = torch.randn((T, d), generator=g, device="cuda").to(BF)
    target = forward(x, teacher, k)[0].float()
    weights = torch.tensor([balance, z], device="cuda")
    history = []
    for _ in range(steps):
        w = {name: t.to(BF) for name, t in w32.items()}
        out, losses, saved = forward(x, w, k)
        diff = out.float() - target
        grads = backward((diff / T).to(BF), weights, saved, w)
        for name in w32:
            w32[name] -= lr * grads[name].float()
        history.append(torch.cat([diff.square().mean()[None], losses]))
        if int(saved["err"].item()) != 0:
            raise M.MoeError(f"device error bits {int(saved['err'].item())}")
    return torch.stack(history).cpu().tolist()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=1024)
    a = ap.parse_args()
    for i, (mse, bal, zl) in enumerate(train(a.steps, a.tokens)):
        print(f"step {i:3d}  mse {mse:.4f}  balance {bal:.4f}  z {zl:.4f}")


if __name__ == "__main__":
    main()
