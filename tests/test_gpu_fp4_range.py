"""Tensor scales at the ends of float32's range: codes and scales of bf16 rows
are the definition's there too (moe_fp4_quantize and its kin)."""
import numpy as np
import pytest
import torch

import dropless_grouped_gemm_gb300 as M
from oracle import fp4 as O

pytestmark = pytest.mark.gpu
BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
DEV = "cuda"
K = 256


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _rows(t, seed=0):
    """bf16 rows of a tensor whose scale is the power of two t: ordinary ones,
    ones with zeros and with every border between two codes, small blocks."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((40, K)) * 400 * np.exp(g.standard_normal((40, 1)))
    x[1, ::3] = 0
    x[2] = 0
    x[2, 7::16] = 0.02                                  # blocks of zeros but one value
    x[3] *= 1e-4
    x[4] = np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], K // 8)
    for i, s in enumerate((2.0 ** -9, 3 * 2.0 ** -9, 2.0 ** -6, 1.125, 1.25, 1.875, 7.0, 13.0, 208.0, 448.0)):
        x[5 + i] = x[4] * s * np.where(np.arange(K) % 5 == 0, -1, 1)
    x[15, ::2] = 0
    x[16] *= 1e4                                        # saturates
    x[17] = 2688
    most = float(torch.finfo(BF).max) / t               # (what bf16 holds at the upper end)
    x = np.clip(x, -most, most)
    with np.errstate(over="ignore", under="ignore"):
        return torch.from_numpy(x * t).float().to(BF)


def _check_rows(q, byte_of, code, byte):
    got = O.unpack(q.cpu().numpy()).reshape(code.shape)
    zero = O.code_values(code) == 0                     # (the sign of a zero says nothing)
    np.testing.assert_array_equal(np.where(zero, got & 7, got), np.where(zero, 0, code))
    np.testing.assert_array_equal(byte_of, byte)


@pytest.mark.parametrize("e", [-126, -125, -120, -119, -118, -117, -110, -101, -100, -99, -95, -94, -93, 93, 94, 95, 100, 101, 110, 117])
def test_powers_of_two(e):
    t = 2.0 ** e
    x = _rows(t)
    assert torch.isfinite(x).all()
    ts = torch.tensor([t], device=DEV)
    code, byte = O.quantize(_f64(x), "nvfp4", t)
    at = O.scale_place([0, 40], K, "nvfp4")
    q, s = M.fp4_quantize(x.to(DEV), scale=ts)
    _check_rows(q, s.cpu().numpy()[at], code, byte)
    # the gather, each row once and in both of its ways
    por = torch.arange(40, dtype=I32, device=DEV)
    off = torch.tensor([0, 40], dtype=I32, device=DEV)
    for inverse in (None, por):
        q, s = M.fp4_permute(x.to(DEV), por, 1, off, scale=ts, row_of_pair=inverse)
        _check_rows(q, s.cpu().numpy()[at], code, byte)
    # weights along either index
    w = torch.zeros(1, 64, K, dtype=BF)
    w[0, :40] = x
    wc, wb = O.quantize(_f64(w[0]), "nvfp4", t)
    wat = O.scale_place([0, 64], K, "nvfp4")
    for along, src in (("cols", w), ("rows", w.transpose(1, 2).contiguous())):
        q, s = M.fp4_quantize_weights(src.to(DEV), along=along, scale=ts)
        _check_rows(q[0], s.cpu().numpy()[wat], wc, wb)


def test_the_scales_of_tiny_and_huge_tensors():
    """moe_fp4_tensor_scale's own scales of them, used."""
    for size in (1e-38, 3e-37, 1e-34, 1e-31, 1e28, 1e34):
        x = torch.from_numpy(np.random.default_rng(3).standard_normal((40, K)) * size).float().to(BF)
        x[3, ::2] = 0
        ts = M.fp4_tensor_scale(x.to(DEV))
        t = O.tensor_scale(_f64(x))
        assert float(ts) == t
        code, byte = O.quantize(_f64(x), "nvfp4", t)
        q, s = M.fp4_quantize(x.to(DEV), scale=ts)
        _check_rows(q, s.cpu().numpy()[O.scale_place([0, 40], K, "nvfp4")], code, byte)


@pytest.mark.parametrize("t", [1.7e-38, 3e-36, 1.1e-28, 6e-29, 3e28, 1.2e38])
def test_scales_that_are_no_powers_of_two(t):
    """The oracle's, but where a quotient lies within 2^-22 of a border."""
    tf = float(np.float32(t))
    g = np.random.default_rng(1)
    x = torch.from_numpy(np.clip(g.standard_normal((40, K)) * 300 * tf, -3.3e38, 3.3e38)).float().to(BF)
    x[1, ::2] = 0
    v = _f64(x)
    code, byte = O.quantize(v, "nvfp4", tf)
    q, s = M.fp4_quantize(x.to(DEV), scale=torch.tensor([t], device=DEV))
    sb = s.cpu().numpy()[O.scale_place([0, 40], K, "nvfp4")]
    a = np.abs(v).reshape(40, -1, 16).max(-1) / (6 * tf)
    mids = (O.E4M3[1:] + O.E4M3[:-1]) / 2
    assert ((sb == byte) | (np.abs(a[..., None] / mids - 1) < 2.0 ** -22).any(-1)).all()
    with np.errstate(divide="ignore", invalid="ignore"):
        u = np.abs(v) / np.repeat(O.scale_values(sb, "nvfp4") * tf, 16, -1)
    halves = (O.MAGNITUDES[1:] + O.MAGNITUDES[:-1]) / 2
    near = (np.abs(u[..., None] / halves - 1) < 2.0 ** -22).any(-1)
    same = O.code_values(O.unpack(q.cpu().numpy())) == O.code_values(code)
    assert (same | near | np.repeat(sb != byte, 16, -1)).all()


@pytest.mark.parametrize("rows", [20, 9000])
def test_zero_outputs_of_a_product_stay_zero(rows):
    """A 4-bit output whose scale is so small that a block's scale times it
    has no reciprocal: zeros are zeros all the same."""
    x = torch.zeros(rows, 512, dtype=BF, device=DEV)
    w = M.fp4_quantize_weights(torch.randn(1, 1024, 512, device=DEV).to(BF), along="cols")
    bias = torch.zeros(1, 1024, dtype=BF, device=DEV)
    bias[0, 5::16] = 2.0 ** -133
    t = torch.tensor([2.0 ** -126], device=DEV)
    (q, s), _, err = M.fp4_linear(M.fp4_quantize(x), None, w, bias=bias, out_dtype="fp4", out_scale=t)
    v = M.fp4_dequantize((q, s), scale=t, dtype=F32)
    keep = torch.ones(1024, dtype=torch.bool, device=DEV)
    keep[5::16] = False
    assert int(err) == 0 and (v[:, keep] == 0).all()


@pytest.mark.parametrize("e", [-126, -100, -60, 60, 100, 117])
def test_nan_and_infinity(e):
    """They mark their block and no other, whatever the scale."""
    t = 2.0 ** e
    x = _rows(t)
    x[20, 5], x[20, 40], x[21, 100], x[22] = float("nan"), float("inf"), -float("inf"), float("nan")
    code, byte = O.quantize(_f64(x), "nvfp4", t)
    at = O.scale_place([0, 40], K, "nvfp4")
    w = torch.zeros(1, 64, K, dtype=BF)
    w[0, :40] = x
    wq, ws = M.fp4_quantize_weights(w.transpose(1, 2).contiguous().to(DEV), along="rows", scale=torch.tensor([t], device=DEV))
    for q, sb in ((M.fp4_quantize(x.to(DEV), scale=torch.tensor([t], device=DEV))), (wq[0, :40], ws)):
        sb = sb.cpu().numpy()[O.scale_place([0, 64], K, "nvfp4")[:40] if q.data_ptr() == wq.data_ptr() else at]
        np.testing.assert_array_equal(sb, byte)
        got = O.unpack(q.cpu().numpy())
        good = np.repeat(byte != 0x7F, 16, -1)
        assert (byte == 0x7F).sum() == 3 + K // 16
        assert ((O.code_values(got) == O.code_values(code)) | ~good).all()
