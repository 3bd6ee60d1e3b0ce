"""Pins of the oracle's operators around the expert MLP: closed forms, and
every gradient against central differences."""
import numpy as np
import pytest

import oracle as O


def _router(seed, T=11, E=6, k=3):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((T, E))
    idx = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    return rng, z, idx


def test_balanced_router_has_loss_one():
    T, E, k = 12, 4, 2
    z = np.zeros((T, E))
    idx = np.stack([[(t + j) % E for j in range(k)] for t in range(T)]).astype(np.int32)
    r = O.router_loss(z, idx)
    assert r["counts"].tolist() == [[6] * 4] and r["n_valid"].tolist() == [12]
    assert abs(r["loss"][0] - 1.0) < 1e-14
    assert abs(r["loss"][1] - np.log(E) ** 2) < 1e-13


def test_collapsed_router_has_loss_e_over_k():
    # every token sends its one pair to expert 0 with probability 1
    z = np.full((5, 8), -200.0)
    z[:, 0] = 0.0
    r = O.router_loss(z, np.zeros((5, 1), np.int32))
    assert abs(r["loss"][0] - 8.0) < 1e-12 and r["loss"][1] < 1e-12


def test_masked_empty_and_unrouted_tokens():
    _, z, idx = _router(1)
    z[3] = -np.inf
    idx[5] = -1
    mask = np.ones(11, np.uint8)
    mask[[0, 7]] = 0
    seg = [0, 4, 4, 9]            # an empty sequence, and tokens after the last
    r = O.router_loss(z, idx, seg, mask)
    assert r["n_valid"].tolist() == [2, 0, 4]
    assert r["counts"].sum(axis=1).tolist() == [6, 0, 9]
    g = O.router_loss_bwd(z, idx, [1.0, 1.0], seg_offsets=seg, token_mask=mask)
    assert np.all(g[[0, 3, 7, 9, 10]] == 0) and np.isfinite(g).all() and np.any(g[1] != 0)
    # no token at all
    r = O.router_loss(z, idx, token_mask=np.zeros(11, np.uint8))
    assert r["loss"].tolist() == [0.0, 0.0]


@pytest.mark.parametrize("seg", [None, [0, 4, 4, 10]])
def test_router_gradient_against_differences(seg):
    rng, z, idx = _router(2)
    mask = np.ones(11, np.uint8)
    mask[6] = 0
    dloss = np.array([0.7, 0.3])
    dp = rng.standard_normal(idx.shape)

    def probs(zz):
        s = np.take_along_axis(zz, idx, 1)
        e = np.exp(s - s.max(axis=1, keepdims=True))
        return e / e.sum(axis=1, keepdims=True)

    def f(zz):
        return float(dloss @ O.router_loss(zz, idx, seg, mask)["loss"]) + float((dp * probs(zz)).sum())

    g = O.router_loss_bwd(z, idx, dloss, probs(z), dp, seg, mask)
    h = 1e-5
    for t in range(11):
        for e in range(6):
            a, b = z.copy(), z.copy()
            a[t, e] += h
            b[t, e] -= h
            # central differences: truncation h^2 f'''/6 and rounding 1e-16 / h
            assert abs((f(a) - f(b)) / (2 * h) - g[t, e]) < 1e-8, (t, e)


ACTS = ["none", "relu", "silu", "gelu", "srelu", "swiglu", "geglu"]


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("act", ACTS)
def test_linear_gradient_against_differences(act, layout):
    rng = np.random.default_rng(3)
    off, K, N = [0, 3, 3, 5], 4, 6
    a, B = rng.standard_normal((5, K)), rng.standard_normal((3, K, N))
    if layout == "nk":
        B = np.swapaxes(B, 1, 2).copy()
    bias = rng.standard_normal((3, N))
    n_out = N // 2 if act in ("swiglu", "geglu") else N
    res, dout = rng.standard_normal((5, n_out)), rng.standard_normal((5, n_out))

    def f(a, B, bias):
        return float((dout * O.linear_fwd(a, off, B, act, bias, res, layout)[0]).sum())

    z = O.linear_fwd(a, off, B, act, bias, res, layout)[1]
    assert np.abs(z).min() > 1e-3            # no kink of relu within the step
    dz, da, dB, db = O.linear_bwd(dout, a, off, B, act, z, layout)
    assert np.all(dB[1] == 0) and np.all(db[1] == 0)      # expert without rows
    h = 1e-5
    for x, g, put in ((a, da, lambda v: f(v, B, bias)), (B, dB, lambda v: f(a, v, bias)),
                      (bias, db, lambda v: f(a, B, v))):
        for i in np.ndindex(x.shape):
            p, q = x.copy(), x.copy()
            p[i] += h
            q[i] -= h
            assert abs((put(p) - put(q)) / (2 * h) - g[i]) < 1e-7, i


def test_checkpoint_values_are_within_half_a_code_step():
    rng = np.random.default_rng(4)
    x = O.bf16_round(rng.standard_normal((7, 128)) * np.exp(3 * rng.standard_normal((7, 1))))
    x[2, 32:64] = 0.0
    q, s = O.checkpoint_pack(x)
    v = O.checkpoint_unpack(q, s)
    scale = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=1)
    # normal codes: half of 2^-3 of the value; below 2^-6 scale units: half of
    # 2^-9 units; above 448 units: saturated, at most 64 units (512 - 448)
    bound = np.maximum(np.abs(x) * 2.0 ** -4, scale * 2.0 ** -10)
    bound = np.where(np.abs(x) > 448 * scale, 64 * scale, bound)
    assert np.all(np.abs(v - x) <= bound)
    assert np.all(v[2, 32:64] == 0.0)
    # the values are their own checkpoint
    q2, s2 = O.checkpoint_pack(v)
    assert np.array_equal(O.checkpoint_unpack(q2, s2), v)
