"""4-bit operators past 2^31 elements and bytes, and at many experts: what the
first and the last rows come out as, against the same rows alone."""
import pytest
import torch

import dropless_grouped_gemm_gb300 as M

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
DEV = "cuda"


def _fill(rows, K, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.empty((rows, K), dtype=BF, device=DEV)
    for i in range(0, rows, 1 << 16):
        x[i:i + (1 << 16)] = torch.randn((min(1 << 16, rows - i), K), generator=g, device=DEV)
    return x


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_rows_whose_codes_pass_2_31_bytes(fmt):
    rows, K, N = 540_001, 8192, 64            # 2.2e9 bytes of codes, 4.4e9 values
    x = _fill(rows, K, 1)
    a = M.fp4_quantize(x, fmt=fmt)
    w = M.fp4_quantize_weights(_fill(N, K, 2)[None], fmt=fmt, along="cols")
    out, _, err = M.fp4_linear(a, None, w, fmt=fmt, out_dtype=F32)
    assert int(err) == 0
    tail = 300
    for sl in (slice(0, tail), slice(rows - tail, rows)):
        b = M.fp4_quantize(x[sl].contiguous(), fmt=fmt)
        ref, _, _ = M.fp4_linear(b, None, w, fmt=fmt, out_dtype=F32)
        # another kernel, whose sums may round otherwise: 2^-22 a stage of the magnitude
        assert float((out[sl] - ref).abs().max()) <= (K / 64) * 2.0 ** -22 * float(ref.abs().max()) * 4
    last = M.fp4_dequantize(a, fmt=fmt)[-tail:]
    assert torch.equal(last, M.fp4_dequantize(M.fp4_quantize(x[-tail:].contiguous(), fmt=fmt), fmt=fmt))


def test_outputs_past_2_31_elements():
    rows, K, N = 530_000, 128, 4096           # 2.2e9 outputs
    x, W = _fill(rows, K, 3), _fill(N, K, 4)
    off = torch.tensor([0, 100, 100, rows - 77, rows], dtype=I32, device=DEV)
    w = M.fp4_quantize_weights(W.expand(4, N, K).contiguous(), along="cols")
    a = M.fp4_quantize(x, off)
    out, z, err = M.fp4_linear(a, off, w, act="silu", save_z=True)
    assert int(err) == 0
    sl = slice(rows - 77, rows)
    ref, rz, _ = M.fp4_linear(M.fp4_quantize(x[sl].contiguous()), None, (w[0][:1].contiguous(), M.fp4_quantize_weights(W[None], along="cols")[1]),
                              act="silu", save_z=True)
    assert torch.equal(z[sl], rz) and torch.equal(out[sl], ref)
    del out, z
    (q, s), _, _ = M.fp4_linear(a, off, w, act="silu", out_dtype="fp4")
    v = M.fp4_dequantize((q, s), off)[sl]
    assert float((v.float() - ref.float()).norm() / ref.float().norm()) < 0.2     # 4 bits: a tenth
    assert torch.isfinite(v).all()


def test_weights_past_2_31_values():
    E, N, K = 40, 8192, 8192                  # 2.7e9 values
    W = torch.empty((E, K, N), dtype=BF, device=DEV)
    for e in range(E):
        W[e] = _fill(K, N, e)
    w = M.fp4_quantize_weights(W, along="rows")
    one = M.fp4_quantize_weights(W[-1:].contiguous(), along="rows")
    assert torch.equal(w[0][-1:], one[0])
    x = _fill(16, K, 7)
    off = torch.zeros(E + 1, dtype=I32, device=DEV)
    off[-1] = 16
    out, _, err = M.fp4_linear(M.fp4_quantize(x, off), off, w)
    ref, _, _ = M.fp4_linear(M.fp4_quantize(x), None, one)
    assert int(err) == 0
    assert float((out.float() - ref.float()).abs().max()) <= 2.0 ** -7 * float(ref.float().abs().max())


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("E,most,K,N", [(1024, 600, 1024, 576), (600, 20, 128, 192)])
def test_many_experts(fmt, E, most, K, N):
    """Above the expert count that leaves the pairs' kernel its boxes, and with
    few rows each."""
    g = torch.Generator().manual_seed(E)
    n = torch.randint(0, most, (E,), generator=g)
    n[3] = n[E - 1] = 0
    off = torch.zeros(E + 1, dtype=I32)
    off[1:] = torch.cumsum(n, 0)
    rows = int(off[-1])
    x = _fill(rows, K, 1)
    W = _fill(E * N, K, 2).reshape(E, N, K)
    d = off.to(DEV)
    a, w = M.fp4_quantize(x, d, fmt=fmt), M.fp4_quantize_weights(W, fmt=fmt, along="cols")
    assert (M.fp4_linear_plan(E, rows, K, N, True)[0] == 0) == (most == 600)
    xv, wv = M.fp4_dequantize(a, d, fmt=fmt, dtype=F32), M.fp4_dequantize(w, fmt=fmt, dtype=F32)
    ref = torch.cat([xv[off[e]:off[e + 1]].double() @ wv[e].double().T for e in range(E)])
    mag = torch.cat([xv[off[e]:off[e + 1]].double().abs() @ wv[e].double().abs().T for e in range(E)])
    for dt in (F32, BF):
        out, _, err = M.fp4_linear(a, d, w, fmt=fmt, out_dtype=dt)
        assert int(err) == 0
        tol = (K / 64 + 10) * 2.0 ** -22 * mag + (2.0 ** -8 * ref.abs() if dt is BF else 0)
        assert ((out.double() - ref).abs() <= tol).all()
    out, _, _ = M.fp4_linear(a, d, w, fmt=fmt, act="relu")
    assert ((out.double() - ref.clamp(min=0)).abs() <= (K / 64 + 10) * 2.0 ** -22 * mag + 2.0 ** -8 * ref.abs()).all()
