"""The operators around the expert MLP, as cases that can be timed and compared.

Three families, each in a plain form (elementary torch operations in 32 bits)
and as calls of this framework:

  router loss    the load-balance and z losses of a router with its per-expert
                 counts, and the router's gradient with respect to the logits
  linear         a grouped (or, with one expert, dense) product with bias,
                 activation and residual, and its backward
  checkpoint     activations kept in 8 bits between forward and backward: token
                 rows packed and gathered back, the expert MLP's forward that
                 keeps H in 8 bits, and its backward that reads it
"""
import math

import torch

own = False

DEV = "cuda"
BF = torch.bfloat16
F32 = torch.float32
GATED = ("swiglu", "geglu")


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a short micro-batch of a small router: launch latency
        dict(name="loss_fwd_t512_e64_k2", op="loss_fwd", T=512, E=64, k=2, S=1, mask=False, dt="f32"),
        # a global batch of 64k tokens in 16 packed sequences, some tokens padding
        dict(name="loss_fwd_t65536_e256_k8_s16", op="loss_fwd", T=65536, E=256, k=8, S=16, mask=True, dt="f32"),
        # the router of the Zipf layer, one training step of 4096 tokens
        dict(name="loss_bwd_t4096_e256_k8", op="loss_bwd", T=4096, E=256, k=8, S=1, mask=False, dt="f32"),
        # odd sizes: bf16 logits and gradients (the gate's weight gradient reads them), ragged sequences, padding
        dict(name="loss_bwd_t30011_e60_k4_s7_bf16", op="loss_bwd", T=30011, E=60, k=4, S=7, mask=True, dt="bf16"),
        # one token through a shared expert's first product: the weights' bytes
        dict(name="linear_m1_k7168_n4096_swiglu", op="linear_fwd", E=1, active=1, M=1, K=7168, N=4096, act="swiglu",
             layout="kn", bias=True, residual=False, save_z=False, out="bf16"),
        # decoding 16 tokens, top-8 of 64 experts: the second product, with its bias
        dict(name="linear_m128_e64_k2048_n7168", op="linear_fwd", E=64, active=57, M=128, K=2048, N=7168, act="none",
             layout="kn", bias=True, residual=False, save_z=False, out="bf16"),
        # the router's gate: 4096 tokens to 256 logits in 32 bits
        dict(name="linear_m4096_k7168_n256_f32", op="linear_fwd", E=1, active=1, M=4096, K=7168, N=256, act="none",
             layout="nk", bias=True, residual=False, save_z=False, out="f32"),
        # the balanced layer's first product in training: bias, gate, saved pre-activation
        dict(name="linear_m32768_e8_k8192_n4096_geglu", op="linear_fwd", E=8, active=8, M=32768, K=8192, N=4096, act="geglu",
             layout="kn", bias=True, residual=False, save_z=True, out="bf16"),
        # backward of ragged experts with biases
        dict(name="linear_bwd_m8191_e8_k2048_n4096_swiglu", op="linear_bwd", E=8, active=7, M=8191, K=2048, N=4096, act="swiglu",
             layout="kn", bias=True),
        # forward of ragged experts that keeps H in 8 bits (the codes' values come back with it)
        dict(name="ckpt_mlp_fwd_m8191_e8_d4096_n1024_geglu", op="ckpt_mlp_fwd", E=8, active=7, M=8191, d=4096, n=1024, act="geglu"),
        # the token rows of the Zipf layer, kept in 8 bits, gathered into expert order for the weight gradient, top-8
        dict(name="ckpt_permute_t4096_k8_d7168", op="ckpt_permute", T=4096, k=8, d=7168),
        # backward of ragged experts from H in 8 bits, with the router's gradient
        dict(name="ckpt_mlp_bwd_m16384_e8_d4096_n2048", op="ckpt_mlp_bwd", E=8, active=8, M=16384, d=4096, n=2048, act="swiglu"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _m64(rng, lo, hi):
    """A multiple of 64 in [lo, hi], spread over the logarithm."""
    while True:
        v = _log(rng, lo // 64, hi // 64) * 64
        if v not in (1536, 3072):
            return v


def draw(rng):
    op = rng.choice(["loss_fwd", "loss_bwd", "linear_fwd", "linear_fwd", "linear_bwd", "ckpt_pack", "ckpt_permute",
                     "ckpt_mlp_fwd", "ckpt_mlp_bwd"])
    if op.startswith("loss"):
        E = _log(rng, 2, 1024)
        T = _log(rng, 1, min(65536, 65536 * 256 // E))
        return dict(op=op, T=T + (T == 3072), E=E, k=rng.randint(1, min(E, 10)), S=_log(rng, 1, min(T, 64)), mask=rng.random() < 0.5,
                    dt=rng.choice(["f32", "bf16"]))
    if op == "ckpt_pack":
        T = _log(rng, 1, 16384)
        return dict(op=op, T=T + (T == 3072), d=_m64(rng, 64, 8192))
    if op == "ckpt_permute":
        T = _log(rng, 1, 8192)
        return dict(op=op, T=T + (T == 3072), k=rng.randint(1, 8), d=_m64(rng, 64, 8192))
    M = _log(rng, 1, 16384)
    M += M == 3072
    E = _log(rng, 1, 64)
    active = max(1, min(M, E, rng.randint((E + 1) // 2, E)))
    if op.startswith("ckpt"):
        d, n = _m64(rng, 128, 4096), _m64(rng, 128, 2048)
        act = rng.choice(["swiglu", "geglu", "srelu"])
        while E * d * n > 1 << 27:
            E = (E + 1) // 2
        return dict(op=op, E=E, active=min(active, E), M=M, d=d, n=n, act=act)
    K, N = _m64(rng, 64, 8192), _m64(rng, 64, 8192)
    while E * K * N > 1 << 29:
        E = (E + 1) // 2
    active = min(active, E)
    while M * K * N > (1 << 39 if op == "linear_fwd" else 1 << 38):
        M = (M + 1) // 2
    M += M == 3072
    act = rng.choice(["none", "relu", "silu", "gelu", "srelu", "swiglu", "geglu"])
    if op == "linear_bwd":
        return dict(op=op, E=E, active=min(active, M), M=M, K=K, N=N, act=act, layout=rng.choice(["kn", "nk"]), bias=rng.random() < 0.7)
    return dict(op=op, E=E, active=min(active, M), M=M, K=K, N=N, act=act, layout=rng.choice(["kn", "nk"]), bias=rng.random() < 0.7,
                residual=rng.random() < 0.5, save_z=rng.random() < 0.3, out=rng.choice(["bf16", "bf16", "f32"]))


# ------------------------------------------------------------------ the inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0, dt=BF):
    return (torch.randn(shape, generator=g, device=DEV, dtype=F32) * std).to(dt)


def _weights(g, *shape, std=0.02):
    """bf16 weights, made one leading slice at a time (no 32-bit copy of a large stack)."""
    w = torch.empty(shape, device=DEV, dtype=BF)
    for e in range(shape[0]):
        w[e] = torch.randn(shape[1:], generator=g, device=DEV, dtype=F32).mul_(std)
    return w


def _ragged(M, E, active, seed):
    """Row counts of E experts, `active` of them with at least one row, skewed; and the most rows of one."""
    r = torch.Generator()
    r.manual_seed(seed + 17)
    order = torch.randperm(E, generator=r)[:active]
    share = torch.rand(active, generator=r, dtype=torch.float64) + 0.25
    c = torch.ones(active, dtype=torch.int64)
    extra = M - active
    add = torch.floor(share / share.sum() * extra).to(torch.int64)
    add[: extra - int(add.sum())] += 1
    counts = torch.zeros(E, dtype=torch.int64)
    counts[order] = c + add
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(counts, 0)
    return off.to(DEV), int(counts.max())


def _pow2(e):
    """2^e in 32 bits, from an integer tensor with -126 <= e <= 127 (below: 0)."""
    return ((e.to(torch.int32) + 127).clamp(min=0) << 23).view(F32)


def _quantise(v):
    """Codes (E4M3) and scale bytes (E8M0) of 32-blocks along the last axis of a 32-bit tensor."""
    b = v.reshape(v.shape[0], -1, 32)
    amax = b.abs().amax(-1)
    e = torch.frexp(amax).exponent - 1
    code = torch.where(amax > 0, (e + 119).clamp(0, 254), torch.zeros_like(e))
    q = (b * _pow2(127 - code)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.reshape(v.shape), code.to(torch.uint8)


def _values(q, s):
    """The 32-bit values that codes and scale bytes stand for."""
    b = q.to(F32).reshape(q.shape[0], -1, 32)
    return (b * _pow2(s.to(torch.int32) - 127)[..., None]).reshape(q.shape)


def _router_inputs(c, g, seed):
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    pop = -1.2 * torch.log(torch.arange(1, E + 1, device=DEV, dtype=F32)) * 0.5
    z = torch.randn((T, E), generator=g, device=DEV, dtype=F32) + pop
    idx = torch.topk(z, k, dim=1).indices.to(torch.int32)
    r = torch.Generator()
    r.manual_seed(seed + 3)
    cut = torch.sort(torch.randperm(T, generator=r)[: S - 1] + 1).values if S > 1 else torch.zeros(0, dtype=torch.int64)
    seg = torch.cat([torch.zeros(1, dtype=torch.int64), cut, torch.tensor([T])]).to(torch.int32).to(DEV)
    mask = (torch.rand(T, generator=g, device=DEV) > 0.1).to(torch.uint8) if c["mask"] else None
    if c["dt"] == "bf16":
        z = z.to(BF)
    return z, idx, seg, mask


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op.startswith("loss"):
        z, idx, seg, mask = _router_inputs(case, g, seed)
        s.update(logits=z, idx=idx, seg=seg if case["S"] > 1 else None, mask=mask)
        if op == "loss_bwd":
            sel = torch.gather(z.to(F32), 1, idx.long())
            p = torch.exp(sel - sel.amax(1, keepdim=True))
            s["probs"] = p / p.sum(1, keepdim=True)
            s["dprobs"] = _normal(g, *sel.shape, std=1e-3, dt=F32)
            s["dloss"] = torch.tensor([1e-2, 1e-3], device=DEV)
            loss, counts, lse, n_valid = _loss_fwd(s)
            s["fwd"] = {"counts": counts, "lse": lse, "n_valid": n_valid}
        return s
    if op.startswith("ckpt") and "T" in case:
        T, d = case["T"], case["d"]
        x = _normal(g, T, d) * torch.exp(0.5 * torch.randn((T, 1), generator=g, device=DEV)).to(BF)
        if op == "ckpt_pack":
            s["x"] = x
        else:
            q, sc = _quantise(x.to(F32))
            s["q"], s["s"] = q.view(torch.uint8), sc
            P = T * case["k"]
            s["pair_of_row"] = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
            row = torch.empty(P, dtype=torch.int32, device=DEV)
            row[s["pair_of_row"].long()] = torch.arange(P, dtype=torch.int32, device=DEV)
            s["row_of_pair"] = row
        return s
    M, E = case["M"], case["E"]
    s["offsets"], s["most"] = _ragged(M, E, case["active"], seed)
    if op.startswith("linear"):
        K, N, act = case["K"], case["N"], case["act"]
        n_out = N // 2 if act in GATED else N
        s["a"] = _normal(g, M, K)
        s["B"] = _weights(g, E, K, N) if case["layout"] == "kn" else _weights(g, E, N, K)
        s["bias"] = _normal(g, E, N, std=0.5) if case["bias"] else None
        if op == "linear_bwd":
            s["z"] = _normal(g, M, N, std=1.5) if act != "none" else None
            s["dout"] = _normal(g, M, n_out, std=0.1)
        else:
            s["residual"] = _normal(g, M, n_out) if case["residual"] else None
        return s
    d, n, act = case["d"], case["n"], case["act"]
    n1 = 2 * n if act in GATED else n
    s["x"] = _normal(g, M, d)
    s["W1"], s["W2"] = _weights(g, E, d, n1), _weights(g, E, n, d)
    if op == "ckpt_mlp_bwd":
        q, sc = _quantise(torch.randn((M, n1), generator=g, device=DEV, dtype=F32) * 1.3)
        s["h_q"], s["h_s"] = q.view(torch.uint8), sc
        s["do"] = _normal(g, M, d, std=0.1)
        s["probs"] = torch.rand((M, 1), generator=g, device=DEV)
        s["pair_of_row"] = torch.randperm(M, generator=g, device=DEV).to(torch.int32)
        row = torch.empty(M, dtype=torch.int32, device=DEV)
        row[s["pair_of_row"].long()] = torch.arange(M, dtype=torch.int32, device=DEV)
        s["row_of_pair"] = row
    return s


# ------------------------------------------------------------------ the plain forms

def _segments(s):
    z, c = s["logits"], s["case"]
    T, S = c["T"], c["S"]
    t = torch.arange(T, device=z.device, dtype=torch.int32)
    seg = torch.zeros(T, dtype=torch.int64, device=z.device) if s["seg"] is None else \
        torch.searchsorted(s["seg"][1:].contiguous(), t, right=True)
    return seg, S


def _loss_fwd(s):
    c, z = s["case"], s["logits"].to(F32)
    E, k = c["E"], c["k"]
    seg, S = _segments(s)
    m = z.amax(1, keepdim=True)
    ex = torch.exp(z - m)
    tot = ex.sum(1, keepdim=True)
    lse = (m + torch.log(tot))[:, 0]
    valid = torch.ones_like(lse) if s["mask"] is None else (s["mask"] != 0).to(F32)
    p = ex / tot * valid[:, None]
    sums = torch.zeros((S, E), device=z.device).index_add_(0, seg, p)
    at = (seg[:, None] * E + s["idx"].long()).reshape(-1)
    counts = torch.zeros(S * E, dtype=torch.int32, device=z.device)
    counts.index_add_(0, at, valid.to(torch.int32)[:, None].expand(-1, k).reshape(-1))
    counts = counts.reshape(S, E)
    n_valid = torch.zeros(S, dtype=torch.int32, device=z.device).index_add_(0, seg, valid.to(torch.int32))
    N = n_valid.sum().to(F32).clamp(min=1)
    bal = ((counts.to(F32) * sums).sum(1) / n_valid.to(F32).clamp(min=1)).sum() * E / (k * N)
    zl = (valid * lse * lse).sum() / N
    return torch.stack([bal, zl]), counts, lse, n_valid


def _loss_bwd(s):
    c, z = s["case"], s["logits"].to(F32)
    E, k = c["E"], c["k"]
    seg, S = _segments(s)
    f = s["fwd"]
    lse = f["lse"][:, None]
    p = torch.exp(z - lse)
    n_s = f["n_valid"].to(F32)
    N = n_s.sum().clamp(min=1)
    w = (s["dloss"][0] * E / (k * N)) * f["counts"].to(F32) / n_s.clamp(min=1)[:, None]
    w = w[seg]
    d = p * (w - (p * w).sum(1, keepdim=True) + 2 * s["dloss"][1] / N * lse)
    if s["mask"] is not None:
        d = d * (s["mask"] != 0).to(F32)[:, None]
    pr, dp = s["probs"], s["dprobs"]
    r = pr * (dp - (pr * dp).sum(1, keepdim=True))
    d = d.scatter_add(1, s["idx"].long(), r)
    return d.to(s["logits"].dtype)


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


_C, _A = math.sqrt(2 / math.pi), 0.044715


def _phi(x, act):
    if act in ("swiglu", "silu"):
        return x * _sigmoid(x)
    if act in ("geglu", "gelu"):
        return x * _sigmoid(2 * _C * (x + _A * x * x * x))
    if act == "relu":
        return x.clamp(min=0)
    if act == "srelu":
        return x.clamp(min=0) * x.clamp(min=0)
    return x


def _dphi(x, act):
    if act in ("swiglu", "silu"):
        g = _sigmoid(x)
        return g * (1 + x * (1 - g))
    if act in ("geglu", "gelu"):
        g = _sigmoid(2 * _C * (x + _A * x * x * x))
        return g + 2 * _C * x * g * (1 - g) * (1 + 3 * _A * x * x)
    if act == "relu":
        return (x > 0).to(x.dtype)
    if act == "srelu":
        return 2 * x.clamp(min=0)
    return torch.ones_like(x)


def _act(z, act):
    return _phi(z[:, 0::2], act) * z[:, 1::2] if act in GATED else _phi(z, act)


def _dact(z, dout, act):
    if act not in GATED:
        return dout * _dphi(z, act)
    g, u = z[:, 0::2], z[:, 1::2]
    return torch.stack([dout * u * _dphi(g, act), dout * _phi(g, act)], dim=2).reshape(z.shape)


class _Rows:
    """The rows of ragged experts as a padded [E, most, .] stack and back."""

    def __init__(self, offsets, most, M):
        dev = offsets.device
        off = offsets.long()
        at = off[:-1, None] + torch.arange(most, device=dev)
        self.ok = at < off[1:, None]
        self.at = torch.where(self.ok, at, torch.zeros_like(at))
        rows = torch.arange(M, device=dev)
        self.e = torch.searchsorted(off[1:].contiguous(), rows, right=True)
        self.pos = rows - off[self.e]

    def out(self, x):
        return x.to(F32)[self.at] * self.ok[..., None].to(F32)

    def back(self, x):
        return x[self.e, self.pos]

    def times(self, x, w):
        return self.back(torch.bmm(self.out(x), w.to(F32)))

    def outer(self, x, y):
        return torch.bmm(self.out(x).transpose(1, 2), self.out(y))


def _linear_fwd(s):
    c = s["case"]
    B = s["B"] if c["layout"] == "kn" else s["B"].transpose(1, 2)
    if c["E"] == 1:
        z = torch.mm(s["a"].to(F32), B[0].to(F32))
        if s["bias"] is not None:
            z = z + s["bias"].to(F32)
    else:
        rows = _Rows(s["offsets"], s["most"], c["M"])
        z = rows.times(s["a"], B)
        if s["bias"] is not None:
            z = z + s["bias"].to(F32)[rows.e]
    out = _act(z, c["act"])
    if s["residual"] is not None:
        out = out + s["residual"].to(F32)
    out = out if c["out"] == "f32" else out.to(BF)
    return {"out": out, "z": z.to(BF)} if c["save_z"] else {"out": out}


def _linear_bwd(s):
    c = s["case"]
    nk = c["layout"] == "nk"
    rows = _Rows(s["offsets"], s["most"], c["M"])
    dout = s["dout"].to(F32)
    dz = dout if s["z"] is None else _dact(s["z"].to(F32), dout, c["act"])
    da = rows.times(dz, s["B"] if nk else s["B"].transpose(1, 2))
    dB = rows.outer(dz, s["a"]) if nk else rows.outer(s["a"], dz)
    r = {"dz": dz.to(BF), "da": da.to(BF), "dB": dB.to(BF)}
    if s["bias"] is not None:
        r["dbias"] = rows.out(dz).sum(1)
    return r


def _mlp_fwd(s):
    c = s["case"]
    rows = _Rows(s["offsets"], s["most"], c["M"])
    h = rows.times(s["x"], s["W1"])
    q, sc = _quantise(h)
    a = _act(h, c["act"])
    return {"h": _values(q, sc).to(BF), "a": a.to(BF), "y": rows.times(a, s["W2"]).to(BF)}


def _mlp_bwd(s):
    c = s["case"]
    rows = _Rows(s["offsets"], s["most"], c["M"])
    h = _values(s["h_q"].view(torch.float8_e4m3fn), s["h_s"])
    p = s["probs"].reshape(-1)[s["pair_of_row"].long()][:, None]
    da = rows.times(s["do"], s["W2"].transpose(1, 2))
    a = _act(h, c["act"])
    ds = (da * a).sum(1)
    dh = _dact(h, p * da, c["act"])
    return {"dh": dh.to(BF), "a_scaled": (p * a).to(BF), "dprobs": ds[s["row_of_pair"].long()][:, None],
            "dx": rows.times(dh, s["W1"].transpose(1, 2)).to(BF), "dW1": rows.outer(s["x"], dh).to(BF),
            "dW2": rows.outer(p * a, s["do"]).to(BF)}


def _plain(s):
    op = s["case"]["op"]
    if op == "loss_fwd":
        loss, counts, lse, n_valid = _loss_fwd(s)
        return {"loss": loss, "counts": counts, "lse": lse, "n_valid": n_valid}
    if op == "loss_bwd":
        return {"dlogits": _loss_bwd(s)}
    if op == "linear_fwd":
        return _linear_fwd(s)
    if op == "linear_bwd":
        return _linear_bwd(s)
    if op == "ckpt_pack":
        q, sc = _quantise(s["x"].to(F32))
        return {"q": q, "s": sc}
    if op == "ckpt_permute":
        v = _values(s["q"].view(torch.float8_e4m3fn), s["s"]).to(BF)
        return {"x_perm": v[(s["pair_of_row"] // s["case"]["k"]).long()]}
    return _mlp_fwd(s) if op == "ckpt_mlp_fwd" else _mlp_bwd(s)


# ------------------------------------------------------------------ the framework's calls

def _framework(s):
    import dropless_grouped_gemm_gb300 as M
    c = s["case"]
    op = c["op"]
    if op == "loss_fwd":
        r = M.router_loss(s["logits"], s["idx"], seg_offsets=s["seg"], token_mask=s["mask"])
        return {"loss": r["loss"], "counts": r["counts"], "lse": r["lse"], "n_valid": r["n_valid"]}
    if op == "loss_bwd":
        return {"dlogits": M.router_loss_bwd(s["logits"], s["idx"], s["fwd"], s["dloss"], probs=s["probs"], dprobs=s["dprobs"],
                                             seg_offsets=s["seg"], token_mask=s["mask"], dtype=s["logits"].dtype)}
    if op == "linear_fwd":
        out, z, _ = M.grouped_linear(s["a"], s["offsets"] if c["E"] > 1 else None, s["B"], act=c["act"], bias=s["bias"],
                                     residual=s["residual"], b_layout=c["layout"], save_z=c["save_z"],
                                     out_dtype=F32 if c["out"] == "f32" else BF)
        return {"out": out, "z": z} if c["save_z"] else {"out": out}
    if op == "linear_bwd":
        dz, da, dB, dbias, _ = M.grouped_linear_bwd(s["dout"], s["a"], s["offsets"], s["B"], act=c["act"], z=s["z"],
                                                    bias=s["bias"] is not None, b_layout=c["layout"])
        r = {"dz": dz, "da": da, "dB": dB}
        if dbias is not None:
            r["dbias"] = dbias
        return r
    if op == "ckpt_pack":
        q, sc = M.checkpoint_pack(s["x"])
        return {"q": q.view(torch.float8_e4m3fn), "s": sc}
    if op == "ckpt_permute":
        return {"x_perm": M.permute_checkpoint(s["q"], s["s"], s["pair_of_row"], c["k"], row_of_pair=s["row_of_pair"])}
    if op == "ckpt_mlp_fwd":
        hq, hs, a, y, _ = M.grouped_mlp_fwd_ckpt(s["x"], s["offsets"], s["W1"], s["W2"], act=c["act"])
        return {"h": M.checkpoint_unpack(hq, hs), "a": a, "y": y}
    dh, a_s, part, dx, dW1, dW2, _ = M.grouped_mlp_bwd_routed_ckpt(
        s["x"], s["h_q"], s["h_s"], s["do"], s["pair_of_row"], s["probs"], s["offsets"], s["W1"], s["W2"], act=c["act"])
    dp = M.router_grad_rows(part, s["row_of_pair"], c["M"], 1)
    return {"dh": dh, "a_scaled": a_s, "dprobs": dp, "dx": dx, "dW1": dW1, "dW2": dW2}


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op.startswith("loss"):
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        w = 2 if case["dt"] == "bf16" else 4
        b = T * E * w + T * k * 4 + T * 4 + S * E * 4 + (T if case["mask"] else 0)
        if op == "loss_bwd":
            b += T * E * w + 2 * T * k * 4
        return {"bytes": b, "flops": 0}
    if op == "ckpt_pack":
        return {"bytes": case["T"] * case["d"] * (2 + 1 + 1 / 32), "flops": 0}
    if op == "ckpt_permute":
        T, k, d = case["T"], case["k"], case["d"]
        return {"bytes": T * d * (1 + 1 / 32) + 2 * T * k * d + 4 * T * k, "flops": 0}
    M, E, act = case["M"], case["E"], case["active"]
    if op == "linear_fwd":
        K, N = case["K"], case["N"]
        n_out = N // 2 if case["act"] in GATED else N
        b = 2 * M * K + 2 * act * K * N + M * n_out * (4 if case["out"] == "f32" else 2)
        b += (2 * M * n_out if case["residual"] else 0) + (2 * M * N if case["save_z"] else 0) + (2 * act * N if case["bias"] else 0)
        return {"bytes": b, "flops": 2 * M * K * N}
    if op == "linear_bwd":
        K, N = case["K"], case["N"]
        n_out = N // 2 if case["act"] in GATED else N
        b = 2 * M * n_out + 2 * M * N * (2 if case["act"] != "none" else 1) + 4 * M * K + 2 * act * K * N + 2 * E * K * N
        return {"bytes": b, "flops": 4 * M * K * N}
    d, n = case["d"], case["n"]
    n1 = 2 * n if case["act"] in GATED else n
    h = M * n1 * (1 + 1 / 32)
    if op == "ckpt_mlp_fwd":
        return {"bytes": 2 * M * d + 2 * act * d * (n1 + n) + h + 2 * M * n + 2 * M * d, "flops": 2 * M * d * (n1 + n)}
    b = 2 * M * d * 3 + h + 2 * act * d * (n1 + n) + 2 * M * (n1 + n) + 2 * E * d * (n1 + n)
    return {"bytes": b, "flops": 4 * M * d * (n1 + n)}


# ------------------------------------------------------------------ in 64 bits, from the definitions

def _two(e):
    """2^e in 64 bits, from an integer tensor."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _e4m3(v):
    """A 64-bit tensor with |v| < 512 rounded to E4M3 values (nearest, ties to even, at most 448)."""
    e = (torch.frexp(v).exponent - 1).clamp(min=-6)
    return (torch.round(v * _two(3 - e)) * _two(e - 3)).clamp(-448, 448)


def _mx_values(v):
    """Scale bytes and the code values (before scaling) of 32-blocks of a 64-bit tensor."""
    b = v.reshape(v.shape[0], -1, 32)
    top = b.abs().max(-1).values
    x = ((torch.frexp(top).exponent - 1).clamp(min=-119) - 8).to(torch.int32)
    x = torch.where(top > 0, x, torch.full_like(x, -127))
    return x + 127, _e4m3(b * _two(-x)[..., None])


def _exact_loss(s, want_bwd):
    c = s["case"]
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    z = s["logits"].double()
    ends = [0, T] if s["seg"] is None else s["seg"].tolist()
    on = torch.ones(T, dtype=torch.bool, device=z.device) if s["mask"] is None else s["mask"] != 0
    lse = torch.logsumexp(z, 1)
    P = torch.exp(z - lse[:, None])
    N = max(1, int(on.sum()))
    bal = 0.0
    counts, n_valid = [], []
    d = torch.zeros_like(z)
    for a, b in zip(ends[:-1], ends[1:]):
        m = on[a:b]
        hits = torch.bincount(s["idx"][a:b][m].reshape(-1).long(), minlength=E)
        n = int(m.sum())
        counts.append(hits)
        n_valid.append(n)
        if n == 0:
            continue
        mean = P[a:b][m].sum(0) / n
        bal = bal + (hits.double() * mean).sum() * E / (k * N)
        if want_bwd:
            g = s["dloss"].double()
            w = g[0] * E / (k * N) * hits.double() / n
            q = P[a:b]
            part = q * (w[None] - (q @ w)[:, None]) + q * (2 * g[1] / N * lse[a:b])[:, None]
            d[a:b] = part * m[:, None].double()
    if want_bwd:
        pr, dp = s["probs"].double(), s["dprobs"].double()
        r = pr * dp - pr * (pr * dp).sum(1, keepdim=True)
        for j in range(k):
            d[torch.arange(T, device=z.device), s["idx"][:, j].long()] += r[:, j]
        return {"dlogits": d}
    zl = (lse[on] ** 2).sum() / N
    return {"loss": torch.stack([torch.as_tensor(bal, device=z.device, dtype=torch.float64), zl]),
            "counts": torch.stack(counts).to(torch.int32), "lse": lse,
            "n_valid": torch.tensor(n_valid, dtype=torch.int32, device=z.device)}


def _gate(x, act):
    """The activation of one 64-bit argument and its derivative."""
    if act in ("swiglu", "silu"):
        f = torch.sigmoid(x)
        return x * f, f + x * f * (1 - f)
    if act in ("geglu", "gelu"):
        u = math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
        t = torch.tanh(u)
        return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 0.134145 * x * x)
    if act == "relu":
        return torch.relu(x), (x > 0).double()
    if act == "srelu":
        return torch.relu(x) ** 2, 2 * torch.relu(x)
    return x, torch.ones_like(x)


def _act64(z, act):
    if act in GATED:
        return _gate(z[:, ::2], act)[0] * z[:, 1::2]
    return _gate(z, act)[0]


def _dact64(z, g, act):
    if act not in GATED:
        return g * _gate(z, act)[1]
    f, df = _gate(z[:, ::2], act)
    out = torch.empty_like(z)
    out[:, ::2] = g * z[:, 1::2] * df
    out[:, 1::2] = g * f
    return out


def exact(case, seed):
    flops = work(case)["flops"]
    if flops > 9e12:
        return None
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("loss"):
        return _exact_loss(s, op == "loss_bwd")
    if op == "ckpt_pack":
        e, v = _mx_values(s["x"].double())
        return {"q": v.reshape(s["x"].shape), "s": e.to(torch.uint8)}
    if op == "ckpt_permute":
        q = s["q"].view(torch.float8_e4m3fn).double().reshape(case["T"], -1, 32)
        v = (q * _two(s["s"].to(torch.int32) - 127)[..., None]).reshape(case["T"], -1)
        return {"x_perm": v[torch.div(s["pair_of_row"], case["k"], rounding_mode="floor").long()]}
    off = s["offsets"].tolist()
    spans = [(e, off[e], off[e + 1]) for e in range(case["E"])]
    if op == "linear_fwd":
        z = torch.empty((case["M"], case["N"]), dtype=torch.float64, device=DEV)
        for e, a, b in spans:
            if b > a:
                w = s["B"][e].double()
                z[a:b] = s["a"][a:b].double() @ (w if case["layout"] == "kn" else w.T)
                if s["bias"] is not None:
                    z[a:b] += s["bias"][e].double()
        out = _act64(z, case["act"])
        if s["residual"] is not None:
            out = out + s["residual"].double()
        return {"out": out, "z": z} if case["save_z"] else {"out": out}
    if op == "linear_bwd":
        g = s["dout"].double()
        dz = g if s["z"] is None else _dact64(s["z"].double(), g, case["act"])
        da = torch.empty((case["M"], case["K"]), dtype=torch.float64, device=DEV)
        dB = torch.zeros(s["B"].shape, dtype=torch.float64, device=DEV)
        db = torch.zeros((case["E"], case["N"]), dtype=torch.float64, device=DEV)
        for e, a, b in spans:
            if b > a:
                w = s["B"][e].double()
                da[a:b] = dz[a:b] @ (w.T if case["layout"] == "kn" else w)
                t = s["a"][a:b].double().T @ dz[a:b]
                dB[e] = t if case["layout"] == "kn" else t.T
                db[e] = dz[a:b].sum(0)
        r = {"dz": dz, "da": da, "dB": dB}
        if s["bias"] is not None:
            r["dbias"] = db
        return r
    M, d, n = case["M"], case["d"], case["n"]
    if op == "ckpt_mlp_fwd":
        h = torch.empty((M, s["W1"].shape[2]), dtype=torch.float64, device=DEV)
        y = torch.empty((M, d), dtype=torch.float64, device=DEV)
        for e, a, b in spans:
            h[a:b] = s["x"][a:b].double() @ s["W1"][e].double()
        act = _act64(h, case["act"])
        for e, a, b in spans:
            y[a:b] = act[a:b] @ s["W2"][e].double()
        x, v = _mx_values(h)
        return {"h": (v * _two(x - 127)[..., None]).reshape(h.shape), "a": act, "y": y}
    h = s["h_q"].view(torch.float8_e4m3fn).double().reshape(M, -1, 32)
    h = (h * _two(s["h_s"].to(torch.int32) - 127)[..., None]).reshape(M, -1)
    p = s["probs"].double().reshape(-1)[s["pair_of_row"].long()]
    act = _act64(h, case["act"])
    dA = torch.empty((M, n), dtype=torch.float64, device=DEV)
    dx = torch.empty((M, d), dtype=torch.float64, device=DEV)
    dW1 = torch.zeros(s["W1"].shape, dtype=torch.float64, device=DEV)
    dW2 = torch.zeros(s["W2"].shape, dtype=torch.float64, device=DEV)
    for e, a, b in spans:
        dA[a:b] = s["do"][a:b].double() @ s["W2"][e].double().T
    dh = _dact64(h, p[:, None] * dA, case["act"])
    for e, a, b in spans:
        dx[a:b] = dh[a:b] @ s["W1"][e].double().T
        dW1[e] = s["x"][a:b].double().T @ dh[a:b]
        dW2[e] = (p[a:b, None] * act[a:b]).T @ s["do"][a:b].double()
    dp = torch.empty((M, 1), dtype=torch.float64, device=DEV)
    dp[s["pair_of_row"].long(), 0] = (dA * act).sum(1)
    return {"dh": dh, "a_scaled": p[:, None] * act, "dprobs": dp, "dx": dx, "dW1": dW1, "dW2": dW2}
