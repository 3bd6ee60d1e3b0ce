"""moe_grouped_linear in every kernel and tile that its choice can take: each
case asserts which kernel serves it, so that another choice cannot empty these
tests unseen.  Tolerances: those of test_gpu_linear.py.  float32 outputs end
their accumulation chains after 64 additions an accumulator, so theirs is
tighter for long reductions: 64 + 2 additions within 2^-22 in a chain, and one
float32 rounding for each chain, accumulator and part of the reduction."""
import numpy as np
import pytest
import torch

import oracle as O
from _helpers import cuda_i32, f64
from test_gpu_linear import _check, _data, _offsets

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32

FEW = [
    # E, M, K, N, kind, (tokens, parts, pair)
    (1, 1, 64, 64, "dense", (16, 1, False)),
    (1, 3, 1024, 192, "dense", (16, 4, False)),
    (1, 9, 2048, 320, "dense", (16, 8, False)),
    (1, 17, 512, 320, "dense", (32, 1, False)),
    (1, 30, 1024, 192, "dense", (32, 4, False)),
    (1, 27, 2048, 128, "dense", (32, 8, False)),
    (1, 40, 640, 192, "dense", (64, 1, False)),
    (1, 63, 1024, 192, "dense", (64, 4, False)),
    (1, 41, 2048, 64, "dense", (64, 8, False)),
    (1, 129, 448, 128, "dense", (128, 1, False)),
    (1, 6000, 2048, 64, "dense", (128, 2, False)),
    (1, 3000, 2048, 128, "dense", (128, 4, False)),
    (1, 130, 2048, 64, "dense", (128, 8, False)),
    (1, 300, 256, 192, "dense", (128, 1, True)),
    (1, 129, 4160, 2048, "dense", (128, 2, True)),
    (1, 131, 2048, 320, "dense", (128, 4, True)),
    (9, 70, 256, 256, "ragged", (16, 1, False)),
    (40, 64, 1024, 64, "ragged", (16, 2, False)),
    (3, 11, 1024, 192, "ragged", (16, 4, False)),
    (2, 5, 2048, 128, "ragged", (16, 8, False)),
    (3, 40, 256, 320, "ragged", (32, 1, False)),
    (8, 100, 1024, 640, "ragged", (32, 2, False)),
    (2, 30, 1024, 192, "ragged", (32, 4, False)),
    (2, 30, 2048, 128, "ragged", (32, 8, False)),
    (4, 100, 384, 128, "ragged", (64, 1, False)),
    (8, 129, 1024, 640, "ragged", (64, 2, False)),
    (2, 63, 1024, 192, "ragged", (64, 4, False)),
    (3, 64, 2048, 192, "ragged", (64, 8, False)),
    (3, 400, 320, 192, "ragged", (128, 1, False)),
    (8, 300, 2048, 640, "ragged", (128, 2, False)),
    (8, 300, 2048, 192, "ragged", (128, 4, False)),
    (2, 129, 2048, 192, "ragged", (128, 8, False)),
    (3, 400, 320, 192, "one", (128, 1, False)),
]


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("E,M,K,N,kind,plan", FEW)
def test_few_row_tiles(E, M, K, N, kind, plan, layout):
    import dropless_grouped_gemm_gb300 as M_
    for i, (act, bias, res, sz, dt) in enumerate([("none", True, False, False, F32),
                                                  ("swiglu", True, True, True, BF),
                                                  ("gelu", False, True, False, BF),
                                                  ("geglu", False, False, True, F32)]):
        assert M_.grouped_linear_plan(E, M, K, N, kind != "dense", dt) == plan
        _check(M_, 200 + i, E, M, K, N, act, layout, kind, bias, res, sz, dt)


# float32 outputs of several chains: parts of K above 32 stages of 64, on CTAs
# with several tiles, in every kind of tile
CHAINS = [
    (1, 1, 2112, 19456, "dense", (16, 1, False)),
    (1, 20, 4160, 19456, "dense", (32, 1, False)),
    (1, 3000, 4160, 2048, "dense", (128, 1, True)),
    (1, 6000, 7168, 64, "dense", (128, 2, False)),
    (30, 200, 4160, 2048, "ragged", (16, 1, False)),
    (30, 1500, 4160, 640, "ragged", (128, 1, False)),
    (8, 140, 7168, 2048, "ragged", (64, 1, False)),
]


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("E,M,K,N,kind,plan", CHAINS)
def test_float32_outputs_over_several_chains(E, M, K, N, kind, plan, layout):
    import dropless_grouped_gemm_gb300 as M_
    assert M_.grouped_linear_plan(E, M, K, N, kind != "dense", F32) == plan
    off = _offsets(kind, E, M, 3)
    a, B, b, _ = _data(30, E, M, K, N, "none", layout, True, False)
    oc = None if off is None else cuda_i32(off)
    out, _, err = M_.grouped_linear(a, oc, B, "none", b, None, layout, out_dtype=F32)
    again, _, _ = M_.grouped_linear(a, oc, B, "none", b, None, layout, out_dtype=F32)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(out, again)
    offs = [0, M] if off is None else off
    # (all rows of the smaller products, some of the larger ones)
    rows = np.unique(np.concatenate([np.linspace(0, M - 1, min(M, 60)).astype(int),
                                     np.clip([o + j for o in offs for j in (-1, 0)], 0, M - 1)]))
    own = np.searchsorted(np.asarray(offs)[1:], rows, side="right")
    want, mag = np.empty((len(rows), N)), np.empty((len(rows), N))
    for e in np.unique(own):
        Be = f64(B[e]) if layout == "kn" else f64(B[e]).T
        at = own == e
        x = f64(a[rows[at]])
        want[at] = x @ Be + f64(b[e])
        mag[at] = np.abs(x) @ np.abs(Be) + np.abs(f64(b[e]))
    parts = K / 2048 + 8 + 2
    got = out[rows].cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - want) <= (66 * 2.0 ** -22 + parts * 2.0 ** -24) * mag + 2.0 ** -24 * np.abs(want))


def _check_relu(M_, seed, E, M, K, N, layout, kind):
    """z within its bound, and out the relu of it bit for bit (rounding keeps
    the sign and the order).  A slope says nothing at the kink, where z may
    round to the other side of 0."""
    off = _offsets(kind, E, M, seed)
    a, B, b, _ = _data(seed, E, M, K, N, "relu", layout, True, False)
    out, z, err = M_.grouped_linear(a, None if off is None else cuda_i32(off), B, "relu", b, None, layout, True)
    torch.cuda.synchronize()
    offs = [0, M] if off is None else off
    want = O.linear_fwd(f64(a), offs, f64(B), "none", f64(b), None, layout)[1]
    mag = O.linear_fwd(np.abs(f64(a)), offs, np.abs(f64(B)), "none", np.abs(f64(b)), None, layout)[1]
    ez = (K / 16 + 16) * 2.0 ** -22 * mag
    assert int(err.item()) == 0 and torch.equal(out, torch.relu(z))
    assert np.all(np.abs(f64(z) - want) <= ez + 2.0 ** -8 * (np.abs(want) + ez))


# the grouped GEMM's tiles: one expert and several, ragged ends, odd widths,
# few rows per expert (the split into two launches), no rows in some
BIG = [
    # E, M, K, N, kind, launches in automatic pair mode
    (1, 8192, 512, 2560, "dense", 1),
    (1, 6000, 64, 1088, "dense", 1),
    (2, 3000, 1024, 4096, "ragged", 1),
    (3, 6000, 512, 2240, "ragged", 1),
    (40, 129, 64, 2048, "ragged", 2),
    (40, 3000, 64, 2176, "one", 2),
]


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("E,M,K,N,kind,launches", BIG)
def test_grouped_gemm_tiles(E, M, K, N, kind, launches, layout):
    import dropless_grouped_gemm_gb300 as M_
    assert M_.grouped_linear_plan(E, M, K, N, kind != "dense", BF)[0] == 0
    for i, (act, bias, res, sz) in enumerate([("none", True, True, False), ("swiglu", True, True, True),
                                              ("gelu", False, False, True), ("geglu", False, True, False),
                                              ("relu", True, False, True)]):
        if act == "relu":
            _check_relu(M_, 300 + i, E, M, K, N, layout, kind)
        else:
            _check(M_, 300 + i, E, M, K, N, act, layout, kind, bias, res, sz, BF)
        assert M_.last_launch_count() == launches


@pytest.mark.parametrize("mode", [0, 2])
@pytest.mark.parametrize("E,M,K,N,kind", [(1, 6000, 64, 1088, "dense"), (2, 3000, 1024, 4096, "ragged"),
                                          (40, 3000, 64, 2176, "one")])
def test_grouped_gemm_tiles_of_either_size(E, M, K, N, kind, mode):
    import dropless_grouped_gemm_gb300 as M_
    before = M_.set_pair_mma(mode)
    try:
        _check(M_, 310, E, M, K, N, "swiglu", "kn", kind, True, True, True, BF)
        _check(M_, 311, E, M, K, N, "silu", "nk", kind, True, True, False, BF)
    finally:
        M_.set_pair_mma(before)


@pytest.mark.parametrize("act", ["relu", "swiglu"])
@pytest.mark.parametrize("E,M,K,N", [(2, 3000, 1024, 4096), (40, 1000, 64, 2048)])
def test_rows_outside_experts_and_residual_in_place(E, M, K, N, act):
    import dropless_grouped_gemm_gb300 as M_
    assert M_.grouped_linear_plan(E, M, K, N, True, BF)[0] == 0
    a, B, b, r = _data(33, E, M, K, N, act, "kn", True, True)
    off = _offsets("ragged", E, M - 7, 5)
    want, _, err = M_.grouped_linear(a, cuda_i32(off), B, act, b, r)
    want = want.clone()
    want[M - 7:] = r[M - 7:]
    out = r.clone()
    M_.grouped_linear(a, cuda_i32(off), B, act, b, out, out=out, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(out, want)


def test_special_values_stay_in_their_rows_of_grouped_gemm_tiles():
    import dropless_grouped_gemm_gb300 as M_
    E, M, K, N = 2, 3000, 1024, 4096
    assert M_.grouped_linear_plan(E, M, K, N, True, BF)[0] == 0
    a, B, b, _ = _data(34, E, M, K, N, "relu", "kn", True, False)
    off = cuda_i32([0, 1111, M])
    clean, _, _ = M_.grouped_linear(a, off, B, "relu", b)
    a = a.clone()
    bad = [0, 127, 1110, 1111, M - 1]
    a[bad, 5] = float("nan")
    out, _, _ = M_.grouped_linear(a, off, B, "relu", b)
    torch.cuda.synchronize()
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert torch.isnan(out[bad]).all() and torch.equal(out[keep], clean[keep])


def test_bad_offsets_in_grouped_gemm_tiles():
    import dropless_grouped_gemm_gb300 as M_
    E, M, K, N = 3, 3000, 1024, 4096
    assert M_.grouped_linear_plan(E, M, K, N, True, BF)[0] == 0
    a, B, b, _ = _data(35, E, M, K, N, "none", "kn", True, False)
    for off in ([0, M, M // 2, M], [0, 1500, 700, M + 5], [2, 3, 4, M]):
        fixed = np.maximum.accumulate(np.clip(off, 0, M))
        want, _, _ = M_.grouped_linear(a, cuda_i32(fixed), B, "none", b)
        out, _, err = M_.grouped_linear(a, cuda_i32(off), B, "none", b)
        torch.cuda.synchronize()
        assert int(err.item()) == M_.DEV_BAD_OFFSETS
        assert torch.equal(out[fixed[0]:fixed[-1]], want[fixed[0]:fixed[-1]])


def test_plan_refusals():
    import dropless_grouped_gemm_gb300 as M_
    for args in ((0, 8, 64, 64, True), (2, 8, 64, 64, False), (1, 0, 64, 64, False), (1, 8, 96, 64, False)):
        with pytest.raises(M_.MoeError):
            M_.grouped_linear_plan(*args)
    with pytest.raises(M_.MoeError):
        M_.grouped_linear_plan(1, 8, 64, 64, False, torch.float16)
