"""Router losses of a contiguous part of a batch, which begins at any row: the
results of a copy of it, bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,out_dtype", [(torch.float32, torch.float32), (torch.float32, torch.bfloat16),
                                             (torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16)])
@pytest.mark.parametrize("E", [4, 7, 8, 33, 60, 250, 1023])
def test_a_part_of_a_batch(E, dtype, out_dtype):
    import dropless_grouped_gemm_gb300 as M
    T, k = 80, 2
    g = torch.Generator(device="cuda").manual_seed(E)
    z = torch.randn((T, E), generator=g, device="cuda").to(dtype)
    idx = z.float().topk(k).indices.int()
    p = torch.rand((T, k), generator=g, device="cuda")
    dp = torch.randn((T, k), generator=g, device="cuda")
    dl = torch.tensor([1.0, 0.5], device="cuda")
    whole = torch.full((T, E), 3.0, dtype=out_dtype, device="cuda")
    for lo in (1, 2, 3, 5):
        part = [t[lo:lo + 61] for t in (z, idx, p, dp)]
        copy = [t.clone() for t in part]
        fa, fb = M.router_loss(*part[:2]), M.router_loss(*copy[:2])
        ga = whole[lo:lo + 61]
        M.router_loss_bwd(part[0], part[1], fa, dl, part[2], part[3], dlogits=ga)
        gb = M.router_loss_bwd(copy[0], copy[1], fb, dl, copy[2], copy[3], dtype=out_dtype)
        torch.cuda.synchronize()
        for n in ("loss", "counts", "lse", "n_valid"):
            assert torch.equal(fa[n], fb[n]), n
        assert torch.equal(ga, gb)
        assert (whole[:lo] == 3.0).all() and (whole[lo + 61:] == 3.0).all()
        whole.fill_(3.0)
