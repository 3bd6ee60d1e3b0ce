"""Product with bias, activation and residual (moe_grouped_linear) and its
backward against the oracle.

Tolerances.  z: products of bf16 values are exact in float32; the tensor
cores add K / 16 groups into a float32 accumulator, each addition within
2^-22 of the running magnitude, and a split reduction adds up to 8 partials:
|dz| <= (K / 16 + 16) 2^-22 sum |a| |B|, plus the bias's rounding.  The
activation moves that by its slope (taken at z, plus 0.5 for its change over
the step; gated: both factors) and its own arithmetic (a sigmoid through a
fast exponential: 2^-18 of the magnitudes).  One rounding of the output:
2^-8 of it in bf16, 2^-24 in float32."""
import numpy as np
import pytest
import torch

import oracle as O
import workloads as W
from _helpers import assert_rms_close, cuda_i32, f64

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "silu", "gelu", "srelu", "swiglu", "geglu"]


def _offsets(kind, E, M, seed=0):
    if kind == "dense":
        return None
    rng = np.random.default_rng(seed)
    if kind == "one":                       # all rows in one expert, the others empty
        c = np.zeros(E, int)
        c[E // 2] = M
    else:
        c = rng.multinomial(M, rng.dirichlet(np.ones(E) * 0.7))
        c[0] += c[-1]
        c[-1] = 0                           # at least one expert has no rows
    return np.concatenate([[0], np.cumsum(c)]).astype(np.int32)


def _data(seed, E, M, K, N, act, layout, bias, residual):
    n_out = N // 2 if act in ("swiglu", "geglu") else N
    a = W.normal((max(M, 1), K), (seed, W.X, 0), 1.0, "cuda")[:M]
    B = W.normal((E, K, N) if layout == "kn" else (E, N, K), (seed, W.W2, 1), 0.05, "cuda")
    b = W.normal((E, N), (seed, W.W2, 2), 0.5, "cuda") if bias else None
    r = W.normal((max(M, 1), n_out), (seed, W.X, 3), 1.0, "cuda")[:M] if residual else None
    return a, B, b, r


def _slope(z, act):
    """|d act| per output for unit changes of z, and the output's magnitude."""
    if act in ("swiglu", "geglu"):
        g, u = z[:, ::2], z[:, 1::2]
        return np.abs(u) * (np.abs(O.dphi(g, act)) + 0.5) + np.abs(O.phi(g, act)) + 0.5, np.abs(g * u)
    return np.abs(O.linear_dact(z, np.ones_like(z), act)) + (0.0 if act in ("none", "relu") else 0.5), np.abs(z) + z * z


def _check(M_, seed, E, M, K, N, act, layout, kind, bias, residual, save_z, dtype):
    off = _offsets(kind, E, M, seed)
    a, B, b, r = _data(seed, E, M, K, N, act, layout, bias, residual)
    out, z, err = M_.grouped_linear(a, None if off is None else cuda_i32(off), B, act, b, r, layout,
                                    save_z, out_dtype=dtype)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    offs = [0, M] if off is None else off
    want, wz = O.linear_fwd(f64(a), offs, f64(B), act, None if b is None else f64(b),
                            None if r is None else f64(r), layout)
    absz = O.linear_fwd(np.abs(f64(a)), offs, np.abs(f64(B)), "none",
                        None if b is None else np.abs(f64(b)), None, layout)[1]
    ez = (K / 16 + 16) * 2.0 ** -22 * absz
    s, mag = _slope(wz, act)
    eo = s * (np.maximum(ez[:, ::2], ez[:, 1::2]) if act in ("swiglu", "geglu") else ez)
    eo = eo + (0 if act in ("none", "relu") else 2.0 ** -18) * mag
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    got = f64(out) if dtype == torch.bfloat16 else out.cpu().numpy().astype(np.float64)
    assert got.shape == want.shape and np.isfinite(got).all()
    assert np.all(np.abs(got - want) <= eo + step * (np.abs(want) + eo))
    if save_z:
        assert np.all(np.abs(f64(z) - wz) <= ez + 2.0 ** -8 * (np.abs(wz) + ez))
    else:
        assert z is None


# the few-row kernel: every tile width, with and without a split reduction,
# odd row counts, half column tiles, both layouts
FEW = [
    # E, M, K, N, kind
    (1, 1, 64, 64, "dense"),
    (1, 1, 2048, 256, "dense"),        # split over 8
    (1, 5, 1024, 192, "dense"),        # a column tile half past N
    (1, 17, 512, 320, "dense"),
    (1, 40, 640, 128, "dense"),
    (1, 129, 448, 256, "dense"),       # two token tiles of 128
    (1, 300, 256, 192, "dense"),       # three token tiles: the last pair has one
    (1, 1000, 512, 256, "dense"),
    (6, 6, 512, 192, "ragged"),
    (9, 70, 256, 256, "ragged"),
    (4, 200, 384, 128, "ragged"),
    (40, 700, 128, 64, "one"),         # 44 tiles of 16 in one expert
    (300, 64, 192, 128, "ragged"),     # most experts empty
    (1024, 40, 64, 64, "ragged"),      # as many experts as there may be
]
# the 128 x 256-tile kernel: ragged ends, pairs of CTAs and single ones
BIG = [
    (1, 2500, 128, 2048, "dense"),
    (1, 5000, 64, 1088, "dense"),
    (5, 3500, 192, 1344, "ragged"),
    (70, 5000, 64, 640, "ragged"),
]


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("E,M,K,N,kind", FEW + BIG)
def test_products(E, M, K, N, kind, layout):
    import dropless_grouped_gemm_gb300 as M_
    for i, (act, bias, res, sz, dt) in enumerate([("none", True, False, False, torch.float32),
                                                  ("swiglu", True, True, True, torch.bfloat16),
                                                  ("gelu", False, True, False, torch.bfloat16)]):
        _check(M_, 100 + i, E, M, K, N, act, layout, kind, bias, res, sz, dt)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ACTS)
def test_activations(act, dtype):
    import dropless_grouped_gemm_gb300 as M_
    _check(M_, 7, 3, 50, 256, 192, act, "kn", "ragged", True, True, True, dtype)
    _check(M_, 8, 2, 3000, 128, 1664, act, "nk", "ragged", True, True, True, dtype)


@pytest.mark.parametrize("M", [3, 2500])
def test_rows_outside_experts_stay_and_residual_in_place(M):
    import dropless_grouped_gemm_gb300 as M_
    K, N = 128, 2048
    a, B, b, r = _data(3, 2, M, K, N, "relu", "kn", True, True)
    off = cuda_i32([0, M // 2, M - 1])
    want, _, err = M_.grouped_linear(a, off, B, "relu", b, r)
    want = want.clone()
    want[-1] = r[-1]
    out = r.clone()
    M_.grouped_linear(a, off, B, "relu", b, out, out=out, err=err)      # in place
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.equal(out, want)
    again, _, _ = M_.grouped_linear(a, off, B, "relu", b, r)
    assert torch.equal(again[:-1], want[:-1])                            # bitwise rerun


def test_bad_offsets_are_corrected_and_reported():
    import dropless_grouped_gemm_gb300 as M_
    for M, N in ((40, 128), (3000, 2048)):
        a, B, b, r = _data(4, 3, M, 64, N, "none", "kn", True, False)
        dout = W.normal((M, N), (4, W.DO, 0), 1.0, "cuda")
        for off in ([0, M, M // 2, M], [0, 1, 2, M + 5], [2, 3, 4, M], [0, -3, 4, M]):
            o = cuda_i32(off)
            _, _, err = M_.grouped_linear(a, o, B, "none", b)
            _, _, _, _, err2 = M_.grouped_linear_bwd(dout, a, o, B, bias=True)
            torch.cuda.synchronize()
            assert int(err.item()) == M_.DEV_BAD_OFFSETS, off
            assert int(err2.item()) == M_.DEV_BAD_OFFSETS, off


def test_special_values_stay_in_their_rows():
    import dropless_grouped_gemm_gb300 as M_
    a, B, b, _ = _data(5, 1, 20, 128, 128, "relu", "kn", True, False)
    clean, _, _ = M_.grouped_linear(a, None, B, "relu", b)
    a = a.clone()
    a[3, 5] = float("nan")
    a[7] = float("inf")
    out, _, _ = M_.grouped_linear(a, None, B, "relu", b)
    torch.cuda.synchronize()
    assert torch.isnan(out[3]).all() and not torch.isfinite(out[7]).all()
    keep = [i for i in range(20) if i not in (3, 7)]
    assert torch.equal(out[keep], clean[keep])


BWD = [
    (1, 1, 64, 64, "dense"),
    (1, 700, 192, 320, "dense"),
    (5, 900, 128, 256, "ragged"),
    (40, 300, 64, 192, "ragged"),
    (3, 1500, 320, 128, "one"),
]


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("E,M,K,N,kind", BWD)
def test_backward(E, M, K, N, kind, layout):
    import dropless_grouped_gemm_gb300 as M_
    for act in (["none", "swiglu", "relu"] if E != 5 else ACTS):
        off = _offsets(kind, E, M, 2)
        offs = [0, M] if off is None else off
        oc = None if off is None else cuda_i32(off)
        a, B, _, _ = _data(20, E, M, K, N, act, layout, False, False)
        n_out = N // 2 if act in ("swiglu", "geglu") else N
        z = W.normal((M, N), (20, W.X, 5), 1.5, "cuda")
        dout = W.normal((M, n_out), (20, W.DO, 0), 1.0, "cuda")
        zz = None if act == "none" else z
        dz, da, dB, db, err = M_.grouped_linear_bwd(dout, a, oc, B, act, zz, True, layout)
        again = M_.grouped_linear_bwd(dout, a, oc, B, act, zz, True, layout)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        wz, _, _, wdb = O.linear_bwd(f64(dout), f64(a), offs, f64(B), act, f64(z), layout)
        if act == "none":
            assert dz is dout
        else:
            zf, g = f64(z), np.abs(f64(dout))
            if act in ("swiglu", "geglu"):
                # |dz| <= |g| |u| (1 + |z|) for the gate, |g| |z| for the up column
                m = np.empty_like(zf)
                m[:, ::2] = g * np.abs(zf[:, 1::2]) * (1 + np.abs(zf[:, ::2]))
                m[:, 1::2] = g * np.abs(zf[:, ::2])
            else:
                m = g * (1 + np.abs(zf)) * (2 if act == "srelu" else 1)
            assert np.all(np.abs(f64(dz) - wz) <= 2.0 ** -18 * m + 2.0 ** -8 * np.abs(wz)), act
        # a column's sum: its elements' errors and one rounding per addition,
        # at most 16 + 8 in a row block and 1/8 of the blocks and 8 after it
        mag = np.stack([np.abs(wz[offs[e]:offs[e + 1]]).sum(axis=0) for e in range(E)])
        adds = 24 + M / 128 / 8 + 8
        el = 0.0 if act in ("none", "relu") else 2.0 ** -17
        bound = (adds * 2.0 ** -24 + el) * mag + el * np.stack(
            [np.abs(f64(z)[offs[e]:offs[e + 1]]).sum(axis=0) * 4 for e in range(E)])
        assert np.all(np.abs(db.cpu().numpy() - wdb) <= bound + 1e-30), act
        gz = f64(dz)
        assert_rms_close(f64(da), O.grouped_gemm(gz, offs, f64(B), "nk" if layout == "kn" else "kn",
                                                 round_out=False), f"linear {act} da")
        assert_rms_close(f64(dB), O.grouped_wgrad(f64(a), gz, offs, False) if layout == "kn"
                         else O.grouped_wgrad(gz, f64(a), offs, False), f"linear {act} dB")
        for x, y in zip((dz, da, dB, db), again):
            assert torch.equal(x, y)


def test_backward_accumulates():
    import dropless_grouped_gemm_gb300 as M_
    E, M, K, N = 4, 500, 128, 192
    off = _offsets("ragged", E, M, 3)
    a, B, _, _ = _data(21, E, M, K, N, "none", "kn", False, False)
    dout = W.normal((M, N), (21, W.DO, 0), 1.0, "cuda")
    _, _, dB, db, _ = M_.grouped_linear_bwd(dout, a, cuda_i32(off), B, bias=True)
    dB0 = W.normal((E, K, N), (21, W.DY, 0), 1.0, "cuda")
    db0 = torch.randn((E, N), device="cuda")
    dB1, db1 = dB0.clone(), db0.clone()
    M_.grouped_linear_bwd(dout, a, cuda_i32(off), B, dB=dB1, dbias=db1, accumulate_dw=True)
    torch.cuda.synchronize()
    assert torch.equal(db1, db0 + db)
    want = f64(dB0) + O.grouped_wgrad(f64(a), f64(dout), off, False)
    assert_rms_close(f64(dB1), want, "linear dB accumulated")
    e = E - 1
    assert off[e] == off[e + 1] and torch.equal(dB1[e], dB0[e]) and torch.equal(db1[e], db0[e])


def test_no_rows():
    import dropless_grouped_gemm_gb300 as M_
    a, B, b, _ = _data(6, 2, 0, 64, 128, "none", "kn", True, False)
    out, _, _ = M_.grouped_linear(a, cuda_i32([0, 0, 0]), B, "none", b)
    assert out.shape == (0, 128)
    _, da, dB, db, _ = M_.grouped_linear_bwd(out, a, cuda_i32([0, 0, 0]), B, bias=True)
    torch.cuda.synchronize()
    assert da.shape == (0, 64) and not dB.any() and not db.any()
    # rows, but none in an expert
    a, B, b, _ = _data(6, 2, 9, 64, 128, "none", "kn", True, False)
    dout = W.normal((9, 128), (6, W.DO, 0), 1.0, "cuda")
    out = torch.full((9, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    M_.grouped_linear(a, cuda_i32([0, 0, 0]), B, "none", b, out=out)
    _, _, dB, db, _ = M_.grouped_linear_bwd(dout, a, cuda_i32([0, 0, 0]), B, bias=True)
    torch.cuda.synchronize()
    assert (out == 7.0).all() and not dB.any() and not db.any()


def test_captures_into_a_graph_on_another_stream():
    import dropless_grouped_gemm_gb300 as M_
    a, B, b, r = _data(9, 1, 3, 1024, 256, "swiglu", "kn", True, True)
    want, _, _ = M_.grouped_linear(a, None, B, "swiglu", b, r)
    out, err = torch.zeros_like(want), torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        M_.grouped_linear(a, None, B, "swiglu", b, r, out=out, err=err)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_a_stream_of_its_own_without_waiting():
    """Calls given a side stream while the current one is busy, with scratch
    and error words of their own: the results of the current stream's calls."""
    import dropless_grouped_gemm_gb300 as M_
    E, M, K, N = 3, 400, 128, 256
    off = cuda_i32(_offsets("ragged", E, M, 4))
    a, B, b, _ = _data(23, E, M, K, N, "silu", "kn", True, False)
    dout = W.normal((M, N), (23, W.DO, 0), 1.0, "cuda")
    want, z, _ = M_.grouped_linear(a, off, B, "silu", b, save_z=True)
    wb = M_.grouped_linear_bwd(dout, a, off, B, "silu", z, True)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    busy = torch.empty(1 << 26, device="cuda")
    for _ in range(4):
        busy.fill_(1.0)                                   # the current stream has work queued
        got, _, err = M_.grouped_linear(a, off, B, "silu", b, z=z.clone(), stream=None)
        st.wait_stream(torch.cuda.current_stream())
        gb = M_.grouped_linear_bwd(dout, a, off, B, "silu", z, True, stream=st)
        junk = torch.full((1 << 20,), float("nan"), device="cuda")   # would land in freed scratch
        st.synchronize()
        assert int(gb[-1].item()) == 0 and int(err.item()) == 0
        assert torch.equal(got, want)
        for x, y in zip(gb[:4], wb[:4]):
            assert torch.equal(x, y)
        del junk


def test_backward_captures_into_a_graph_on_another_stream():
    import dropless_grouped_gemm_gb300 as M_
    E, M, K, N = 3, 400, 128, 256
    off = cuda_i32(_offsets("ragged", E, M, 4))
    a, B, _, _ = _data(22, E, M, K, N, "swiglu", "kn", False, False)
    z = W.normal((M, N), (22, W.X, 5), 1.5, "cuda")
    dout = W.normal((M, N // 2), (22, W.DO, 0), 1.0, "cuda")
    want = M_.grouped_linear_bwd(dout, a, off, B, "swiglu", z, True)
    bufs = dict(zip(("dz", "da", "dB", "dbias", "err"), (torch.zeros_like(t) for t in want)))
    ws = torch.full((M_.grouped_linear_bwd_workspace_size(E, M, N),), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        M_.grouped_linear_bwd(dout, a, off, B, "swiglu", z, True, workspace=ws, **bufs)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for name, t in zip(bufs, want):
        assert torch.equal(bufs[name], t), name
