"""Activations in 8 bits: packing and unpacking bit for bit against the
oracle's block rule, the gather against packing's values, the forward's codes
against the bf16 H, and the backward bit for bit against the routed backward
on the unpacked H."""
import numpy as np
import pytest
import torch

import oracle as O
import workloads as W
from _helpers import cuda_i32, f64
from test_gpu_routed import CASES, _setup

pytestmark = pytest.mark.gpu


def _rows(seed, rows, cols):
    x = W.normal((rows, cols), (seed, W.X, 0), 1.0, "cuda")
    s = torch.exp2(torch.randint(-20, 20, (rows, cols // 32), device="cuda").float())
    return (x.float().view(rows, -1, 32) * s[..., None]).view(rows, cols).to(torch.bfloat16)


@pytest.mark.parametrize("rows,cols", [(1, 64), (3, 192), (37, 7168), (1000, 320)])
def test_pack_and_unpack_bit_exact(rows, cols):
    import dropless_grouped_gemm_gb300 as M
    x = _rows(rows, rows, cols)
    x[0, :32] = 0.0
    x[-1, 32:64] = 2.0 ** -130                        # below the smallest scale
    q, s = M.checkpoint_pack(x)
    v = M.checkpoint_unpack(q, s)
    torch.cuda.synchronize()
    oq, os_ = O.checkpoint_pack(f64(x))
    assert np.array_equal(s.cpu().numpy(), os_)
    # the sign of a zero code is the oracle's too
    assert np.array_equal(q.cpu().numpy(), oq)
    assert np.array_equal(f64(v), O.bf16_round(O.checkpoint_unpack(oq, os_)))


def test_special_values():
    import dropless_grouped_gemm_gb300 as M
    x = torch.ones((2, 64), dtype=torch.bfloat16, device="cuda")
    x[0, 3] = float("inf")
    x[1, 40] = float("nan")
    x[1, 41] = torch.finfo(torch.bfloat16).max
    q, s = M.checkpoint_pack(x)
    v = M.checkpoint_unpack(q, s)
    torch.cuda.synchronize()
    v = v.float().cpu()
    assert v[0, 3] == float("inf") and (v[0, :3] == 0).all()
    assert torch.isnan(v[1, 40]) and torch.isfinite(v[1, 41]) and v[1, 41] > 2.0 ** 126
    assert (v[0, 32:] == 1).all() and (v[1, :32] == 1).all()


@pytest.mark.parametrize("T,k,d,align,E", [(1, 1, 64, 1, 2), (100, 2, 192, 32, 5), (333, 8, 7168, 1, 16)])
def test_gather(T, k, d, align, E):
    import dropless_grouped_gemm_gb300 as M
    rng = np.random.default_rng(T)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    idx[T // 2, 0] = -1                               # an unrouted pair
    r = M.route_offsets(cuda_i32(idx), E, align)
    q, s = M.checkpoint_pack(_rows(T, T, d))
    v = M.checkpoint_unpack(q, s)
    want = M.permute(v, r["pair_of_row"], k)
    a = M.permute_checkpoint(q, s, r["pair_of_row"], k)
    b = M.permute_checkpoint(q, s, r["pair_of_row"], k, row_of_pair=r["row_of_pair"])
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)


@pytest.mark.parametrize("act", ["swiglu", "geglu", "srelu"])
@pytest.mark.parametrize("E,M_rows,d,n,ragged", [(3, 200, 128, 64, True), (4, 2300, 192, 320, True),
                                                 (40, 900, 64, 128, True), (1, 1, 64, 64, False)])
def test_forward(E, M_rows, d, n, ragged, act):
    import dropless_grouped_gemm_gb300 as M
    rng = np.random.default_rng(E)
    c = rng.multinomial(M_rows, rng.dirichlet(np.ones(E))) if ragged else np.array([M_rows])
    off = cuda_i32(np.concatenate([[0], np.cumsum(c)]))
    x = W.normal((M_rows, d), (31, W.X, 0), 1.0, "cuda")
    W1 = (W.w1_plain(31, E, d, n, 0.1, "cuda") if act == "srelu" else W.w1_interleaved(31, E, d, n, 0.1, "cuda"))
    W2 = W.w2(31, E, n, d, 0.1, "cuda")
    h, a, y, err = M.grouped_mlp_fwd(x, off, W1, W2, act, save_h=True)
    hq, hs, a2, y2, err2 = M.grouped_mlp_fwd_ckpt(x, off, W1, W2, act)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and int(err2.item()) == 0
    assert torch.equal(a, a2) and torch.equal(y, y2)
    # h is the float32 H rounded to bf16: its block's largest value may have
    # been rounded up to a power of two, and only then may the scales differ
    hf, sb = f64(h), hs.cpu().numpy().astype(int)
    _, want = O.checkpoint_pack(hf)
    want = want.astype(int)
    top = np.abs(hf).reshape(M_rows, -1, 32).max(axis=-1)
    pow2 = np.frexp(top)[0] == 0.5
    assert np.all((sb == want) | (pow2 & (sb == want - 1)))
    v = O.checkpoint_unpack(hq.cpu().numpy(), sb)
    scale = np.repeat(np.ldexp(1.0, sb - 127), 32, axis=1)
    # half a code step of the float32 H (saturated: 64 scale units), half a
    # bf16 step between it and h
    bound = np.maximum(np.abs(hf) * 2.0 ** -4, scale * 2.0 ** -10) * (1 + 2.0 ** -7)
    bound = np.where(np.abs(hf) > 448 * scale, 65 * scale, bound) + np.abs(hf) * 2.0 ** -8
    assert np.all(np.abs(v - hf) <= bound)


@pytest.mark.parametrize("act", ["swiglu", "geglu", "srelu"])
@pytest.mark.parametrize("name,E,T,k,d,n,align", CASES, ids=[c[0] for c in CASES])
def test_backward_equals_routed_backward_on_the_unpacked_h(name, E, T, k, d, n, align, act):
    M, idx, probs, r, ro, x, H, tok_dO, do_perm, W1, W2 = _setup(act, E, T, k, d, n, align, 61)
    pt = torch.from_numpy(probs).cuda().view(-1)
    q, s = M.checkpoint_pack(H)
    v = M.checkpoint_unpack(q, s)
    want = M.grouped_mlp_bwd_routed(x, v, do_perm, r["pair_of_row"], pt, r["offsets"], W1, W2, act)
    got = M.grouped_mlp_bwd_routed_ckpt(x, q, s, do_perm, r["pair_of_row"], pt, r["offsets"], W1, W2, act)
    torch.cuda.synchronize()
    assert int(got[-1].item()) == 0
    R = int(ro["offsets"][-1])
    for nm, a, b in zip(("dh", "a_scaled", "ds_part", "dx"), want, got):
        assert torch.equal(a[:R], b[:R]), nm
    assert torch.equal(want[4], got[4]) and torch.equal(want[5], got[5])
    # accumulating twice
    dW1, dW2 = got[4].clone(), got[5].clone()
    M.grouped_mlp_bwd_routed_ckpt(x, q, s, do_perm, r["pair_of_row"], pt, r["offsets"], W1, W2, act,
                                  dW1=dW1, dW2=dW2, accumulate_dw=True)
    ref1, ref2 = want[4].clone(), want[5].clone()
    M.grouped_mlp_bwd_routed(x, v, do_perm, r["pair_of_row"], pt, r["offsets"], W1, W2, act,
                             dW1=ref1, dW2=ref2, accumulate_dw=True)
    torch.cuda.synchronize()
    assert torch.equal(dW1, ref1) and torch.equal(dW2, ref2)


@pytest.mark.parametrize("mode", [0, 2])
def test_pair_modes_agree(mode):
    import dropless_grouped_gemm_gb300 as M
    M, idx, probs, r, ro, x, H, tok_dO, do_perm, W1, W2 = _setup("swiglu", 3, 700, 2, 128, 192, 1, 62)
    pt = torch.from_numpy(probs).cuda().view(-1)
    q, s = M.checkpoint_pack(H)

    def run():
        f = M.grouped_mlp_fwd_ckpt(x, r["offsets"], W1, W2, "swiglu")
        b = M.grouped_mlp_bwd_routed_ckpt(x, q, s, do_perm, r["pair_of_row"], pt, r["offsets"], W1, W2)
        torch.cuda.synchronize()
        return f[:4] + b[:6]

    want = run()
    old = M.set_pair_mma(mode)
    try:
        got = run()
    finally:
        M.set_pair_mma(old)
    R = int(ro["offsets"][-1])
    for a, b in zip(want, got):
        assert torch.equal(a[:R], b[:R]) if a.dim() == 2 else torch.equal(a, b)
