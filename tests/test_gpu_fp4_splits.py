"""The few-row product in 4 bits with every part count of its reduction and
every kind of output (moe_fp4_linear)."""
import numpy as np
import pytest
import torch

import dropless_grouped_gemm_gb300 as M
from oracle import fp4 as O
from test_gpu_fp4_linear import Case, _check, _gated

pytestmark = pytest.mark.gpu
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
DEV = "cuda"
FMT = ["nvfp4", "mxfp4"]
TAILS = {0: (128, 512, 1152, 2048, 4096, 8192), 64: (64, 448, 1088, 2112, 4160)}


def _sizes(split, tail):
    """Up to three of the sizes, the smallest to the largest, that the kernel choice splits so."""
    takes = [(m, k, n) for k in (512, 1024, 2048, 4096, 7168) for n in TAILS[tail] for m in (1, 16, 40, 64, 100, 200)
             if M.fp4_linear_plan(1, m, k, n, False) == (64, split)]
    assert takes
    return sorted({takes[0], takes[len(takes) // 2], takes[-1]})


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("act,tail", [("swiglu", 0), ("silu", 64), ("none", 0)])
@pytest.mark.parametrize("split", [1, 2, 4, 8])
def test_four_bit_outputs(split, act, tail, fmt):
    for m, k, n in _sizes(split, tail):
        c = Case([0, m], k, n, fmt, dense=True)
        n_out = n // 2 if _gated(act) else n
        t = torch.tensor([0.25], device=DEV) if fmt == "nvfp4" else None
        out = (torch.full((m, n_out // 2), 0xAB, dtype=U8, device=DEV),
               torch.full((M.fp4_scale_bytes(m, 1, n_out, fmt),), 0xCD, dtype=U8, device=DEV))
        (q, s), _, err = c.run(act=act, bias=c.bias, out=out, out_scale=t)
        full, _, _ = c.run(act=act, bias=c.bias, out_dtype=F32)
        assert int(err) == 0
        # the codes of the float32 outputs, but where a quotient lies within 2^-21 of
        # a border (a reciprocal's and a product's rounding)
        v = full.double().cpu().numpy()
        tf = 1.0 if t is None else float(t)
        code, byte = O.quantize(v, fmt, tf)
        at = O.scale_place([0, m], n_out, fmt)
        sb = s.cpu().numpy()
        np.testing.assert_array_equal(sb[at], byte)
        with np.errstate(divide="ignore", invalid="ignore"):
            u = np.abs(v) / np.repeat(O.scale_values(byte, fmt) * tf, O.BLOCK[fmt], -1)
        halves = (O.MAGNITUDES[1:] + O.MAGNITUDES[:-1]) / 2
        near = (np.abs(u[..., None] / halves - 1) < 2.0 ** -21).any(-1)
        assert ((O.code_values(O.unpack(q.cpu().numpy())) == O.code_values(code)) | near).all()
        free = np.ones(sb.size, bool)
        free[at.reshape(-1)] = False
        assert (sb[free] == 0xCD).all()


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("split", [1, 2, 4, 8])
def test_float32_and_bf16_outputs(split, fmt):
    for tail in TAILS:
        for m, k, n in _sizes(split, tail):
            c = Case([0, m], k, n, fmt, dense=True)
            _check(c, act="gelu", out_dtype=F32, residual=True, save_z=True)
            _check(c, act="none", bias=False)


@pytest.mark.parametrize("fmt", FMT)
def test_ragged_tiles_of_every_split(fmt):
    """Experts of 0, 1, 64 and 65 rows (a tile's second half of a scale tile),
    with 4-bit outputs and whatever part count these sizes get."""
    seen = set()
    for k, n in ((512, 256), (2048, 128), (4096, 128), (7168, 64), (7168, 1024), (2048, 4096)):
        for offsets in ([0, 1], [0, 0, 64, 65], [0, 65, 65, 130, 131], [0, 3, 133, 134, 200]):
            c = Case(offsets, k, n, fmt, extra=3)
            plan = M.fp4_linear_plan(c.E, c.rows, k, n, True)
            if plan[0] == 0:
                continue
            seen.add(plan[1])
            full, _, err = c.run(act="silu", bias=c.bias, out_dtype=F32)
            (q, s), _, _ = c.run(act="silu", bias=c.bias, out_dtype="fp4")
            assert int(err) == 0
            ref = M.fp4_quantize(full.to(BF), c.off, fmt=fmt)         # (the layout; values to a bf16 rounding)
            got = M.fp4_dequantize((q, s), c.off, fmt=fmt, dtype=F32)[:c.last]
            want = M.fp4_dequantize(ref, c.off, fmt=fmt, dtype=F32)[:c.last]
            # a 4-bit step is at most half of a block's largest value over 3: two
            # quantisations of values 2^-8 apart differ by no more than one
            top = full[:c.last].abs().reshape(c.last, -1, O.BLOCK[fmt]).amax(-1).repeat_interleave(O.BLOCK[fmt], 1)
            assert ((got - want).abs() <= top * 0.5 + 1e-30).all()
            _check(c, act="silu", save_z=True)
    assert len(seen) >= 2
