"""The 4-bit formats against the float64 oracle: quantisation, permute,
weights, the values read back, tensor scales (moe_fp4_*)."""
import numpy as np
import pytest
import torch

import dropless_grouped_gemm_gb300 as M
from oracle import fp4 as O

pytestmark = pytest.mark.gpu
BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
DEV = "cuda"
FMT = ["nvfp4", "mxfp4"]


def _rows(rows, K, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, K), generator=g) * std * torch.exp(torch.randn((rows, 1), generator=g))
    return x.to(BF)


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _poisoned(rows, E, K, fmt):
    return (torch.full((rows, K // 2), 0xAB, dtype=U8, device=DEV),
            torch.full((M.fp4_scale_bytes(rows, E, K, fmt),), 0xCD, dtype=U8, device=DEV))


def _check(q, s, x, offsets, K, fmt, t=1.0):
    """Codes and scales exactly the oracle's, nothing else written."""
    q, s = q.cpu().numpy(), s.cpu().numpy()
    last = int(offsets[-1])
    code, byte = O.quantize(x[:last], fmt, t)
    got = O.unpack(q[:last])
    zero = O.code_values(code) == 0                     # (the sign of a zero says nothing)
    np.testing.assert_array_equal(np.where(zero, got & 7, got), np.where(zero, 0, code))
    at = O.scale_place(offsets, K, fmt)
    np.testing.assert_array_equal(s[at], byte)
    assert (q[last:] == 0xAB).all()
    free = np.ones(s.size, bool)
    free[at.reshape(-1)] = False
    assert (s[free] == 0xCD).all()


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("rows,K", [(1, 64), (3, 128), (31, 192), (129, 320), (128, 512), (300, 576), (5, 1088), (2, 7168)])
def test_dense(fmt, rows, K):
    x = _rows(rows, K, rows + K)
    q, s = M.fp4_quantize(x.to(DEV), fmt=fmt, out=_poisoned(rows, 1, K, fmt))
    _check(q, s, _f64(x), [0, rows], K, fmt)
    for dt in (BF, F32):
        v = M.fp4_dequantize((q, s), fmt=fmt, dtype=dt)
        np.testing.assert_array_equal(_f64(v), O.values(*O.quantize(_f64(x), fmt), fmt))


OFFSETS = [[0, 7], [0, 5, 5, 133, 300], [0, 0, 0, 130, 131, 131], [0, 127, 255, 383, 384], [0, 0], [0, 256, 256, 600]]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("offsets", OFFSETS)
def test_ragged(fmt, offsets):
    K, rows = 192, offsets[-1] + 9
    x = _rows(rows, K, 3)
    off = torch.tensor(offsets, dtype=I32, device=DEV)
    E = len(offsets) - 1
    err = torch.zeros(1, dtype=I32, device=DEV)
    q, s = M.fp4_quantize(x.to(DEV), off, fmt=fmt, out=_poisoned(rows, E, K, fmt), err=err)
    _check(q, s, _f64(x), offsets, K, fmt)
    out = torch.full((rows, K), 7.0, dtype=BF, device=DEV)
    M.fp4_dequantize((q, s), off, fmt=fmt, out=out, err=err)
    last = offsets[-1]
    np.testing.assert_array_equal(_f64(out)[:last], O.values(*O.quantize(_f64(x)[:last], fmt), fmt))
    assert (out[last:] == 7).all() and int(err) == 0


@pytest.mark.parametrize("t", [2.0 ** -11, 0.25, 4.0])
def test_tensor_scales(t):
    x = _rows(40, 256, 5, std=t)
    ts = torch.tensor([t], device=DEV)
    q, s = M.fp4_quantize(x.to(DEV), fmt="nvfp4", scale=ts, out=_poisoned(40, 1, 256, "nvfp4"))
    _check(q, s, _f64(x), [0, 40], 256, "nvfp4", t)
    v = M.fp4_dequantize((q, s), scale=ts, dtype=F32)
    np.testing.assert_array_equal(_f64(v), O.values(*O.quantize(_f64(x), "nvfp4", t), "nvfp4", t))


def test_a_tensor_scale_that_is_no_power_of_two():
    """Scales and codes are the oracle's, but where a quotient lies within
    2^-22 (three float32 roundings) of a border."""
    t = 0.0037
    tf = float(np.float32(t))
    x = _rows(200, 512, 6, std=0.1)
    q, s = M.fp4_quantize(x.to(DEV), scale=torch.tensor([t], device=DEV))
    code, byte = O.quantize(_f64(x), "nvfp4", tf)
    at = O.scale_place([0, 200], 512, "nvfp4")
    np.testing.assert_array_equal(s.cpu().numpy()[at], byte)
    u = np.abs(_f64(x)) / np.repeat(O.scale_values(byte, "nvfp4") * tf, 16, -1)
    halves = (O.MAGNITUDES[1:] + O.MAGNITUDES[:-1]) / 2
    near = (np.abs(u[..., None] / halves - 1) < 2.0 ** -22).any(-1)
    got = O.unpack(q.cpu().numpy())
    same = O.code_values(got) == O.code_values(code)
    assert (same | near).all()
    v = M.fp4_dequantize((q, s), scale=torch.tensor([t], device=DEV), dtype=F32)
    ref = O.values(got, byte, "nvfp4", tf)
    assert (np.abs(_f64(v) - ref) <= 2.0 ** -24 * np.abs(ref)).all()


@pytest.mark.parametrize("fmt", FMT)
def test_special_values(fmt):
    x = _rows(12, 256, 8)
    x[0] = 0
    x[1] = -0.0
    x[2, 5], x[2, 77], x[2, 130] = float("nan"), float("inf"), -float("inf")
    x[3] = torch.finfo(BF).max
    x[4] = -torch.finfo(BF).max
    x[5] *= 1e-38
    x[6] = 2.0 ** -133                      # bf16's smallest
    x[7] *= 1e30
    x[8] *= 1e-4                            # E4M3 scales of nvfp4 underflow
    x[9, ::2] = 0
    x[10] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 32).to(BF)      # every border
    x[11] = x[10] * 1.125
    q, s = M.fp4_quantize(x.to(DEV), fmt=fmt, out=_poisoned(12, 1, 256, fmt))
    byte = O.quantize(_f64(x), fmt)[1]
    np.testing.assert_array_equal(s.cpu().numpy()[O.scale_place([0, 12], 256, fmt)], byte)
    v = _f64(M.fp4_dequantize((q, s), fmt=fmt, dtype=F32))
    ref = O.values(*O.quantize(_f64(x), fmt), fmt)
    # (a float32 below 2^-126 may read back as 0)
    small = np.abs(ref) < 2.0 ** -126
    np.testing.assert_array_equal(np.isnan(v), np.isnan(ref))
    assert ((v == ref) | np.isnan(ref) | (small & (np.abs(v) <= 2.0 ** -126))).all()


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("E,R,C", [(1, 64, 64), (3, 128, 192), (2, 192, 320), (4, 64, 256), (1, 512, 64), (5, 256, 128)])
@pytest.mark.parametrize("along", ["rows", "cols"])
def test_weights(fmt, E, R, C, along):
    W = torch.stack([_rows(R, C, e, 0.02 * 4 ** e) for e in range(E)])
    t = M.fp4_tensor_scale(W.to(DEV), per_expert=True) if fmt == "nvfp4" else None
    N, K = (C, R) if along == "rows" else (R, C)
    out = (torch.full((E, N, K // 2), 0xAB, dtype=U8, device=DEV), _poisoned(E * N, E, K, fmt)[1])
    q, s = M.fp4_quantize_weights(W.to(DEV), fmt=fmt, along=along, scale=t, out=out)
    x = _f64(W).transpose(0, 2, 1) if along == "rows" else _f64(W)
    ref = []
    for e in range(E):
        te = 1.0 if t is None else float(t[e])
        if t is not None:
            assert te == O.tensor_scale(x[e])
        code, byte = O.quantize(x[e], fmt, te)
        ref.append(O.values(code, byte, fmt, te))
        got = O.unpack(q[e].cpu().numpy())
        assert (O.code_values(got) == O.code_values(code)).all()
        at = O.scale_place([i * N for i in range(E + 1)], K, fmt)[e * N:(e + 1) * N]
        np.testing.assert_array_equal(s.cpu().numpy()[at], byte)
    v = M.fp4_dequantize((q, s), fmt=fmt, scale=t, dtype=F32)
    np.testing.assert_array_equal(_f64(v), np.stack(ref))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("T,k,E,d,align", [(1, 1, 1, 64, 1), (17, 2, 5, 192, 1), (40, 8, 16, 576, 16), (200, 4, 3, 320, 32),
                                           (9, 33, 40, 128, 1)])
def test_permute(fmt, T, k, E, d, align):
    g = torch.Generator().manual_seed(T)
    idx = torch.stack([torch.randperm(E, generator=g)[:min(k, E)] for _ in range(T)]).to(I32)
    idx[T // 2, 0] = -1
    k = idx.shape[1]
    r = M.route_offsets(idx.to(DEV), E, align, M_cap=T * k + E * (align - 1) + 5)
    x = _rows(T, d, 4).to(DEV)
    rows = r["pair_of_row"].numel()
    ref = M.permute(x, r["pair_of_row"], k)
    offsets = r["offsets"].cpu().numpy()
    t = M.fp4_tensor_scale(x) if fmt == "nvfp4" else None
    for inverse in (None, r["row_of_pair"]):
        q, s = M.fp4_permute(x, r["pair_of_row"], k, r["offsets"], fmt=fmt, scale=t, row_of_pair=inverse,
                             out=_poisoned(rows, E, d, fmt))
        _check(q, s, _f64(ref), offsets, d, fmt, 1.0 if t is None else float(t))


def test_tensor_scale():
    for n in (64, 128, 4096, 64 * 1001):
        x = _rows(1, n, n)[0]
        x[n // 2], x[n - 1] = float("nan"), float("-inf")
        assert float(M.fp4_tensor_scale(x.to(DEV))) == O.tensor_scale(_f64(x))
    assert float(M.fp4_tensor_scale(torch.zeros(64, dtype=BF, device=DEV))) == 1
    x = torch.zeros(3, 64, dtype=BF, device=DEV)
    x[1, 3], x[2, 63] = 2688, -3.0
    assert M.fp4_tensor_scale(x, per_expert=True).tolist() == [1, 1, 2.0 ** -9]
    x[0] = torch.finfo(BF).max
    assert float(M.fp4_tensor_scale(x)) == O.tensor_scale([float(torch.finfo(BF).max)])


def test_offsets_that_are_not_in_order_are_reported():
    x = _rows(300, 128, 1).to(DEV)
    for off in ([0, 200, 100, 300], [0, -5, 100, 300], [3, 100, 200, 300], [0, 100, 200, 400]):
        err = torch.zeros(1, dtype=I32, device=DEV)
        o = torch.tensor(off, dtype=I32, device=DEV)
        q, s = M.fp4_quantize(x, o, err=err)
        assert int(err) == M.DEV_BAD_OFFSETS
        err.zero_()
        v = M.fp4_dequantize((q, s), o, err=err, out=torch.zeros(300, 128, dtype=BF, device=DEV))
        assert int(err) == M.DEV_BAD_OFFSETS
        safe = np.maximum.accumulate(np.clip(off, 0, 300))
        ref = O.values(*O.quantize(_f64(x), "nvfp4"), "nvfp4")
        got = _f64(v)
        np.testing.assert_array_equal(got[safe[0]:safe[-1]], ref[safe[0]:safe[-1]])
        assert (got[:safe[0]] == 0).all()


def test_nothing_to_do():
    x = torch.empty(0, 128, dtype=BF, device=DEV)
    q, s = M.fp4_quantize(x)
    assert q.shape == (0, 64) and M.fp4_dequantize((q, s)).shape == (0, 128)
    off = torch.zeros(4, dtype=I32, device=DEV)
    q, s = M.fp4_permute(x, torch.empty(0, dtype=I32, device=DEV), 2, off)
    assert q.shape == (0, 64)
    q, s = M.fp4_permute(x, torch.full((5,), -1, dtype=I32, device=DEV), 2, off, out=_poisoned(5, 3, 128, "nvfp4"),
                         row_of_pair=torch.empty(0, dtype=I32, device=DEV))
    assert (q == 0xAB).all()                # rows of no expert
