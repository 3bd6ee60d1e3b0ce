"""Routing to experts and the experts' products in 4 bits, as cases that can be timed and compared.

In a plain form (elementary torch operations) and as calls of this framework:

  select   the router's choice: softmax or sigmoid scores, a bias that balances
           the choice alone, groups of experts, renormalised and scaled weights,
           and the gradient of the logits from the weights' gradient
  pack     rows and weights in 4 bits (E2M1 codes; "nvfp4": an E4M3 scale per
           16 values and one float32 scale for the tensor, "mxfp4": an E8M0
           scale per 32 values) and the values read back
  linear   a grouped (or, with one expert, dense) product of rows and weights
           in 4 bits with bias, activation and residual; its backward, whose
           data gradient is a 4-bit product too; and the expert MLP of two
           such products, the hidden activations going from one to the other
           in 4 bits
"""
import math

import torch

own = False

DEV = "cuda"
BF = torch.bfloat16
F32 = torch.float32
F64 = torch.float64
E4M3 = torch.float8_e4m3fn
GATED = ("swiglu", "geglu")


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # decoding 16 tokens: sigmoid scores, a balancing bias, 4 of 8 groups: launch latency
        dict(name="select_t16_e256_k8_sigmoid_bias_g8", op="select", T=16, E=256, k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, best=2, renorm=True, scale=2.5, dt="f32"),
        # the same router over a global batch of 64k tokens
        dict(name="select_t65536_e256_k8_sigmoid_bias_g8", op="select", T=65536, E=256, k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, best=2, renorm=True, scale=2.5, dt="f32"),
        # the router of the Zipf layer, one training step of 4096 tokens
        dict(name="select_bwd_t4096_e256_k8_sigmoid", op="select_bwd", T=4096, E=256, k=8, score="sigmoid", bias=True, groups=1,
             top_groups=1, best=1, renorm=True, scale=1.0, dt="f32"),
        # odd sizes: softmax over all experts, weights left as they are (a dense gradient), bf16 logits and gradients
        dict(name="select_bwd_t30011_e60_k4_softmax_bf16", op="select_bwd", T=30011, E=60, k=4, score="softmax", bias=False, groups=1,
             top_groups=1, best=1, renorm=False, scale=1.0, dt="bf16"),
        # the token rows of the Zipf layer in expert order, top-8, quantised and read back
        dict(name="pack_t4096_k8_d7168_nvfp4", op="pack", T=4096, k=8, E=256, d=7168, fmt="nvfp4", scaled=False),
        # one step's cast of a layer's weights, stored with the reduction index outermost
        dict(name="pack_w_e8_k8192_n4096_mxfp4", op="pack_w", E=8, rows=8192, cols=4096, along="rows", fmt="mxfp4"),
        # one token through a shared expert's first product: the weights' bytes, and latency
        dict(name="linear_m1_k7168_n4096_swiglu_nvfp4", op="linear", E=1, active=1, M=1, K=7168, N=4096, act="swiglu", bias=True,
             residual=False, save_z=False, out="bf16", fmt="nvfp4"),
        # decoding 16 tokens, top-8 of 64 experts: the second product, with its bias
        dict(name="linear_m128_e64_k2048_n7168_mxfp4", op="linear", E=64, active=57, M=128, K=2048, N=7168, act="none", bias=True,
             residual=False, save_z=False, out="bf16", fmt="mxfp4"),
        # the balanced layer's first product in training: bias, gate, saved pre-activation
        dict(name="linear_m32768_e8_k8192_n4096_geglu_nvfp4", op="linear", E=8, active=8, M=32768, K=8192, N=4096, act="geglu", bias=True,
             residual=False, save_z=True, out="bf16", fmt="nvfp4"),
        # backward of ragged experts with biases
        dict(name="linear_bwd_m8191_e8_k2048_n4096_swiglu_nvfp4", op="linear_bwd", E=8, active=7, M=8191, K=2048, N=4096, act="swiglu",
             bias=True, fmt="nvfp4"),
        # backward of a shared expert's second product on a short micro-batch
        dict(name="linear_bwd_m512_k2048_n4096_mxfp4", op="linear_bwd", E=1, active=1, M=512, K=2048, N=4096, act="none", bias=False,
             fmt="mxfp4"),
        # serving a prefill batch: the whole expert MLP in 4 bits, ragged experts
        dict(name="mlp_m8191_e8_d4096_n1024_swiglu_nvfp4", op="mlp", E=8, active=7, M=8191, d=4096, n=1024, act="swiglu", fmt="nvfp4"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _m64(rng, lo, hi):
    """A multiple of 64 in [lo, hi], spread over the logarithm."""
    return _log(rng, lo // 64, hi // 64) * 64


def draw(rng):
    op = rng.choice(["select", "select", "select_bwd", "pack", "pack_w", "linear", "linear", "linear_bwd", "mlp"])
    if op.startswith("select"):
        score, bias = rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5
        groups = rng.choice([1, 1, 2, 4, 8])
        E = _log(rng, 2, 1024 // groups) * groups
        top_groups = rng.randint((groups + 1) // 2, groups)
        best = rng.randint(1, min(2, E // groups))
        k = rng.randint(1, min(E // groups * top_groups, 10))
        return dict(op=op, T=_log(rng, 1, min(65536, 65536 * 256 // E)), E=E, k=k, score=score, bias=bias, groups=groups,
                    top_groups=top_groups, best=best, renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]), dt=rng.choice(["f32", "bf16"]))
    fmt = rng.choice(["nvfp4", "mxfp4"])
    if op == "pack":
        E = _log(rng, 1, 256)
        k = rng.randint(1, min(8, E))
        return dict(op=op, T=_log(rng, 1, 8192), k=k, E=E, d=_m64(rng, 64, 8192 if k <= 4 else 4096), fmt=fmt,
                    scaled=fmt == "nvfp4" and rng.random() < 0.5)
    if op == "pack_w":
        rows, cols = _m64(rng, 64, 8192), _m64(rng, 64, 8192)
        E = _log(rng, 1, max(1, (1 << 28) // (rows * cols)))
        return dict(op=op, E=E, rows=rows, cols=cols, along=rng.choice(["rows", "cols"]), fmt=fmt)
    M, E = _log(rng, 1, 16384), _log(rng, 1, 64)
    active = max(1, min(M, E, rng.randint((E + 1) // 2, E)))
    if op == "mlp":
        d, n, act = _m64(rng, 128, 4096), _m64(rng, 128, 2048), rng.choice(["swiglu", "geglu", "srelu"])
        while E * d * n > 1 << 27:
            E = (E + 1) // 2
        return dict(op=op, E=E, active=min(active, E), M=M, d=d, n=n, act=act, fmt=fmt)
    K, N = _m64(rng, 64, 8192), _m64(rng, 64, 8192)
    while E * K * N > 1 << 29:
        E = (E + 1) // 2
    while M * K * N > (1 << 39 if op == "linear" else 1 << 38):
        M = (M + 1) // 2
    active = min(active, E, M)
    act = rng.choice(["none", "relu", "silu", "gelu", "srelu", "swiglu", "geglu"])
    if op == "linear_bwd":
        return dict(op=op, E=E, active=active, M=M, K=K, N=N, act=act, bias=rng.random() < 0.7, fmt=fmt)
    return dict(op=op, E=E, active=active, M=M, K=K, N=N, act=act, bias=rng.random() < 0.7, residual=rng.random() < 0.5,
                save_z=rng.random() < 0.3, out=rng.choice(["bf16", "bf16", "f32"]), fmt=fmt)


# ------------------------------------------------------------------ the inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0, dt=BF):
    return (torch.randn(shape, generator=g, device=DEV, dtype=F32) * std).to(dt)


def _ragged(M, E, active, seed):
    """Row counts of E experts, `active` of them with at least one row, skewed; and the most rows of one."""
    r = torch.Generator()
    r.manual_seed(seed + 17)
    order = torch.randperm(E, generator=r)[:active]
    share = torch.rand(active, generator=r, dtype=F64) + 0.25
    extra = M - active
    add = torch.floor(share / share.sum() * extra).to(torch.int64)
    add[: extra - int(add.sum())] += 1
    counts = torch.zeros(E, dtype=torch.int64)
    counts[order] = 1 + add
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(counts, 0)
    return off.to(DEV), int(counts.max())


def _block(fmt):
    return 16 if fmt == "nvfp4" else 32


def _scale_bytes(s, fmt, E):
    """The scale bytes [E, rows, blocks] of equally long experts in the order that a product takes: tiles of 128 rows
    x 4 blocks, row r and block b of a tile at byte (r % 32) * 16 + (r // 32) * 4 + b; expert e's tiles begin with
    number e * rows // 128 + e."""
    _, rows, nb = s.shape
    rt, ct = -(-rows // 128), -(-nb // 4)
    full = torch.zeros((E, rt * 128, ct * 4), dtype=torch.uint8, device=s.device)
    full[:, :rows, :nb] = s
    t = full.reshape(E, rt, 4, 32, ct, 4).permute(0, 1, 4, 3, 2, 5).reshape(E, rt, ct * 512)
    out = torch.zeros((E * rows // 128 + E, ct * 512), dtype=torch.uint8, device=s.device)
    at = torch.arange(E, device=s.device)
    at = (at * rows // 128 + at)[:, None] + torch.arange(rt, device=s.device)
    out[at.reshape(-1)] = t.reshape(E * rt, ct * 512)
    return out.reshape(-1)


def _weights4(g, E, N, K, fmt, std=0.02):
    """Weights [E, N, K] held in 4 bits, blocks along K: packed codes, scale bytes and the experts' scales as a
    program keeps them, and the values (codes times block scales, exact in bf16) that they stand for."""
    q = torch.empty((E, N, K // 2), dtype=torch.uint8, device=DEV)
    s = torch.empty((E, N, K // _block(fmt)), dtype=torch.uint8, device=DEV)
    t = torch.ones(E, dtype=F32, device=DEV)
    val = torch.empty((E, N, K), dtype=BF, device=DEV)
    for e in range(E):
        w = torch.randn((N, K), generator=g, device=DEV, dtype=F32).mul_(std).to(BF).to(F32)
        if fmt == "nvfp4":
            t[e] = _tensor_scale(w)
        code, sb, sv = _quantise(w, fmt, t[e])
        mag = code.abs()
        idx = torch.where(mag < 2, 2 * mag, torch.where(mag < 4, mag + 2, mag / 2 + 4)).to(torch.uint8) + (code < 0).to(torch.uint8) * 8
        q[e] = idx[:, 0::2] + idx[:, 1::2] * 16
        s[e] = sb
        val[e] = (code.reshape(N, -1, _block(fmt)) * sv[..., None]).reshape(N, K).to(BF)
    return {"q": q, "s": _scale_bytes(s, fmt, E), "t": t if fmt == "nvfp4" else None, "val": val}


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op.startswith("select"):
        T, E, k = case["T"], case["E"], case["k"]
        pop = -0.6 * torch.log(torch.arange(1, E + 1, device=DEV, dtype=F32))
        z = torch.randn((T, E), generator=g, device=DEV, dtype=F32) + pop[torch.randperm(E, generator=g, device=DEV)]
        s["logits"] = z if case["dt"] == "f32" else z.to(BF)
        s["bias"] = _normal(g, E, std=0.05, dt=F32) if case["bias"] else None
        if op == "select_bwd":
            r = _select(s)
            s["idx"], s["probs"] = r["topk_idx"], r["probs"]
            s["dprobs"] = _normal(g, T, k, std=1e-3, dt=F32)
        return s
    fmt = case["fmt"]
    if op == "pack":
        T, k, E = case["T"], case["k"], case["E"]
        x = torch.randn((T, case["d"]), generator=g, device=DEV, dtype=F32)
        x = (x * torch.exp(0.5 * torch.randn((T, 1), generator=g, device=DEV)) * (0.01 if case["scaled"] else 1.0)).to(BF)
        # every token's k experts, then the expert-major rows of the pairs in their order
        idx = torch.topk(torch.rand((T, E), generator=g, device=DEV) - 0.1 * torch.rand(E, generator=g, device=DEV), k, dim=1).indices
        pairs = torch.sort(idx.reshape(-1), stable=True)
        s["x"], s["pair_of_row"] = x, pairs.indices.to(torch.int32)
        s["row_of_pair"] = torch.empty_like(s["pair_of_row"])
        s["row_of_pair"][pairs.indices] = torch.arange(T * k, dtype=torch.int32, device=DEV)
        s["offsets"] = torch.searchsorted(pairs.values, torch.arange(E + 1, device=DEV)).to(torch.int32)
        s["t"] = _tensor_scale(x.to(F32)).reshape(1) if case["scaled"] else None
        return s
    if op == "pack_w":
        s["w"] = torch.empty((case["E"], case["rows"], case["cols"]), device=DEV, dtype=BF)
        for e in range(case["E"]):
            s["w"][e] = torch.randn((case["rows"], case["cols"]), generator=g, device=DEV, dtype=F32).mul_(0.02)
        return s
    M, E = case["M"], case["E"]
    s["offsets"], s["most"] = _ragged(M, E, case["active"], seed)
    if op == "mlp":
        d, n = case["d"], case["n"]
        s["x"] = _normal(g, M, d)
        s["w1"] = _weights4(g, E, 2 * n if case["act"] in GATED else n, d, fmt)
        s["w2"] = _weights4(g, E, d, n, fmt)
        return s
    K, N = case["K"], case["N"]
    n_out = N // 2 if case["act"] in GATED else N
    s["a"] = _normal(g, M, K)
    s["bias"] = _normal(g, E, N, std=0.5) if case["bias"] else None
    if op == "linear_bwd":
        s["w"] = _weights4(g, E, K, N, fmt)     # the copy whose blocks run along N
        s["z"] = _normal(g, M, N, std=1.5) if case["act"] != "none" else None
        s["dout"] = _normal(g, M, n_out, std=0.01)
    else:
        s["w"] = _weights4(g, E, N, K, fmt)
        s["residual"] = _normal(g, M, n_out) if case["residual"] else None
    return s


# ------------------------------------------------------------------ the plain forms

def _pow2(e):
    """2^e in 32 bits, from an integer tensor with -126 <= e <= 127."""
    return ((e.to(torch.int32) + 127) << 23).view(F32)


def _tensor_scale(v):
    """The smallest power of two t with max|v| <= 6 * 448 t (1 for a tensor of zeros)."""
    top = v.abs().max()
    m, e = torch.frexp(top / 2688)
    return torch.where(top > 0, _pow2((e - (m == 0.5).to(e.dtype)).clamp(-126, 127)), torch.ones_like(top))


def _e2m1(u):
    """Rounded to the values of E2M1 (nearest, ties to the even code, at most 6)."""
    a = u.abs().clamp(max=6)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, u)


def _quantise(v, fmt, t):
    """Code values, scale bytes and scale values (without t) of the blocks along the last axis of a 32-bit tensor."""
    b = v.reshape(v.shape[0], -1, _block(fmt))
    amax = b.abs().amax(-1)
    if fmt == "nvfp4":
        s = (amax / (6 * t)).clamp(max=448).to(E4M3)
        sv = s.to(F32)
        d = (sv * t)[..., None]
        return _e2m1(torch.where(d > 0, b / d, torch.zeros_like(b))).reshape(v.shape), s.view(torch.uint8), sv
    byte = torch.where(amax > 0, (torch.frexp(amax).exponent + 124).clamp(0, 254), torch.zeros_like(amax, dtype=torch.int32))
    sv = _pow2((byte - 127).clamp(min=-126))
    return _e2m1(b / sv[..., None]).reshape(v.shape), byte.to(torch.uint8), sv


def _held(v, fmt, t=None):
    """The 32-bit values that a 32-bit tensor keeps in 4 bits."""
    t = 1.0 if t is None else t
    code, _, sv = _quantise(v, fmt, t)
    return (code.reshape(v.shape[0], -1, _block(fmt)) * (sv * t)[..., None]).reshape(v.shape)


def _scores(z, score):
    """In 64 bits: the choice is among values that may lie next to each other."""
    z = z.to(F64)
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    ex = torch.exp(z - z.amax(1, keepdim=True))
    return ex / ex.sum(1, keepdim=True)


def _select(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    p = _scores(s["logits"], c["score"])
    choice = p if s["bias"] is None else p + s["bias"].to(F64)
    if c["top_groups"] < G:
        by = torch.sort(choice.reshape(T, G, E // G), dim=2, descending=True).values[:, :, : c["best"]].sum(2)
        keep = torch.sort(by, dim=1, descending=True, stable=True).indices[:, : c["top_groups"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device=p.device).scatter_(1, keep, True)
        choice = torch.where(kept[:, :, None].expand(T, G, E // G).reshape(T, E), choice, torch.full_like(choice, -math.inf))
    idx = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(p, 1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"topk_idx": idx.to(torch.int32), "probs": (w * c["scale"]).to(F32)}


def _select_bwd(s):
    c, idx = s["case"], s["idx"].long()
    z, w, dw = s["logits"].to(F32), s["probs"], s["dprobs"]
    d = w * dw
    if c["renorm"]:
        d = w * (dw - d.sum(1, keepdim=True) / c["scale"])
    if c["score"] == "sigmoid":
        d = d * (1 - 1 / (1 + torch.exp(-torch.gather(z, 1, idx))))
    out = torch.zeros_like(z).scatter_add(1, idx, d)
    if c["score"] == "softmax" and not c["renorm"]:
        ex = torch.exp(z - z.amax(1, keepdim=True))
        out = out - ex / ex.sum(1, keepdim=True) * d.sum(1, keepdim=True)
    return {"dlogits": out.to(s["logits"].dtype)}


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
        return x[self.at] * self.ok[..., None].to(F32)

    def back(self, x):
        return x[self.e, self.pos]

    def outer(self, x, y):
        return torch.bmm(self.out(x).transpose(1, 2), self.out(y))


def _product(rows, x, w):
    """The rows' product with their expert's weights [E, N, K]."""
    v = w["val"].to(F32)
    v = v if w["t"] is None else v * w["t"][:, None, None]
    if v.shape[0] == 1:
        return torch.mm(x, v[0].T)
    return rows.back(torch.bmm(rows.out(x), v.transpose(1, 2)))


def _linear(s):
    c = s["case"]
    rows = _Rows(s["offsets"], s["most"], c["M"])
    z = _product(rows, _held(s["a"].to(F32), c["fmt"]), s["w"])
    if s["bias"] is not None:
        z = z + s["bias"].to(F32)[rows.e]
    out = _act(z, c["act"])
    if s["residual"] is not None:
        out = out + s["residual"].to(F32)
    out = out if c["out"] == "f32" else out.to(BF)
    return {"out": out, "z": z.to(BF)} if c["save_z"] else {"out": out}


def _linear_bwd(s):
    c = s["case"]
    rows = _Rows(s["offsets"], s["most"], c["M"])
    g = s["dout"].to(F32)
    g = g if s["z"] is None else _dact(s["z"].to(F32), g, c["act"])
    dz = g.to(BF)                   # what both products take
    d = dz.to(F32)
    t = _tensor_scale(d) if c["fmt"] == "nvfp4" else None
    r = {"dz": dz, "da": _product(rows, _held(d, c["fmt"], t), s["w"]).to(BF), "dB": rows.outer(s["a"].to(F32), d).to(BF)}
    if s["bias"] is not None:
        r["dbias"] = rows.out(g).sum(1)
    return r


def _mlp(s):
    c = s["case"]
    rows = _Rows(s["offsets"], s["most"], c["M"])
    h = _act(_product(rows, _held(s["x"].to(F32), c["fmt"]), s["w1"]), c["act"])
    return {"y": _product(rows, _held(h, c["fmt"]), s["w2"]).to(BF)}


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "select":
        return _select(s)
    if op == "select_bwd":
        return _select_bwd(s)
    if op == "pack":
        x = s["x"][torch.div(s["pair_of_row"], c["k"], rounding_mode="floor").long()]
        return {"values": _held(x.to(F32), c["fmt"], s["t"]).to(BF)}
    if op == "pack_w":
        w = s["w"].to(F32)
        w = w.transpose(1, 2).contiguous() if c["along"] == "rows" else w
        return {"values": _held(w.reshape(-1, w.shape[2]), c["fmt"]).reshape(w.shape).to(BF)}
    return _linear(s) if op == "linear" else _linear_bwd(s) if op == "linear_bwd" else _mlp(s)


# ------------------------------------------------------------------ the framework's calls

def _framework(s):
    import dropless_grouped_gemm_gb300 as M
    c = s["case"]
    op = c["op"]
    if op == "select":
        idx, probs = M.router_select(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"], top_groups=c["top_groups"],
                                     group_best=c["best"], renorm=c["renorm"], scale=c["scale"])
        return {"topk_idx": idx, "probs": probs}
    if op == "select_bwd":
        return {"dlogits": M.router_select_bwd(s["logits"], s["idx"], s["probs"], s["dprobs"], score=c["score"], renorm=c["renorm"],
                                               scale=c["scale"], dtype=s["logits"].dtype)}
    fmt = c["fmt"]
    if op == "pack":
        x4 = M.fp4_permute(s["x"], s["pair_of_row"], c["k"], s["offsets"], fmt=fmt, scale=s["t"], row_of_pair=s["row_of_pair"])
        return {"values": M.fp4_dequantize(x4, s["offsets"], fmt=fmt, scale=s["t"])}
    if op == "pack_w":
        w4 = M.fp4_quantize_weights(s["w"], fmt=fmt, along=c["along"])
        return {"values": M.fp4_dequantize(w4, fmt=fmt)}
    off = s["offsets"] if c["E"] > 1 else None
    if op == "mlp":
        w1, w2 = s["w1"], s["w2"]
        x4 = M.fp4_quantize(s["x"], off, fmt=fmt)
        h4, _, err = M.fp4_linear(x4, off, (w1["q"], w1["s"]), fmt=fmt, act=c["act"], w_scale=w1["t"], out_dtype="fp4")
        y, _, _ = M.fp4_linear(h4, off, (w2["q"], w2["s"]), fmt=fmt, w_scale=w2["t"], err=err)
        return {"y": y}
    w = s["w"]
    if op == "linear":
        a4 = M.fp4_quantize(s["a"], off, fmt=fmt)
        out, z, _ = M.fp4_linear(a4, off, (w["q"], w["s"]), fmt=fmt, act=c["act"], bias=s["bias"], residual=s["residual"], w_scale=w["t"],
                                 save_z=c["save_z"], out_dtype=F32 if c["out"] == "f32" else BF)
        return {"out": out, "z": z} if c["save_z"] else {"out": out}
    dz, da, dB, dbias, _ = M.fp4_linear_bwd(s["dout"], s["a"], off, (w["q"], w["s"]), fmt=fmt, act=c["act"], z=s["z"], w_scale=w["t"],
                                            bias=s["bias"] is not None)
    r = {"dz": dz, "da": da, "dB": dB}
    if dbias is not None:
        r["dbias"] = dbias
    return r


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op.startswith("select"):
        T, E, k = case["T"], case["E"], case["k"]
        w = 2 if case["dt"] == "bf16" else 4
        if op == "select":
            return {"bytes": T * E * w + 8 * T * k + (4 * E if case["bias"] else 0), "flops": 0}
        dense = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": T * E * w * (2 if dense else 1) + 12 * T * k + (w * T * k if case["score"] == "sigmoid" else 0), "flops": 0}
    h = 0.5 + 1 / _block(case["fmt"])       # bytes of a value and its share of a scale
    if op == "pack":
        n = case["T"] * case["d"]
        return {"bytes": 2 * n + n * case["k"] * (2 * h + 2) + 8 * case["T"] * case["k"], "flops": 0}
    if op == "pack_w":
        return {"bytes": case["E"] * case["rows"] * case["cols"] * (2 + 2 * h + 2), "flops": 0}
    M, E, act = case["M"], case["E"], case["active"]
    if op == "mlp":
        d, n = case["d"], case["n"]
        n1 = 2 * n if case["act"] in GATED else n
        return {"bytes": 2 * M * d + act * d * (n1 + n) * h + 2 * M * d, "flops": 2 * M * d * (n1 + n)}
    K, N = case["K"], case["N"]
    n_out = N // 2 if case["act"] in GATED else N
    if op == "linear":
        b = 2 * M * K + act * K * N * h + M * n_out * (4 if case["out"] == "f32" else 2)
        b += (2 * M * n_out if case["residual"] else 0) + (2 * M * N if case["save_z"] else 0) + (2 * act * N if case["bias"] else 0)
        return {"bytes": b, "flops": 2 * M * K * N}
    b = 2 * M * n_out + 2 * M * N * (2 if case["act"] != "none" else 0) + 4 * M * K + act * K * N * h + 2 * E * K * N
    return {"bytes": b + (4 * E * N if case["bias"] else 0), "flops": 4 * M * K * N}


# ------------------------------------------------------------------ in 64 bits, from the definitions

_HALVES = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)      # between the codes 0, 0.5, 1, 1.5, 2, 3, 4, 6


def _code64(u):
    """The number of the E2M1 magnitude nearest to a 64-bit tensor's, the even one of two as near."""
    a = u.abs()
    n = torch.zeros_like(a, dtype=torch.int64)
    for j, half in enumerate(_HALVES):
        n += (a >= half) if j % 2 else (a > half)
    return n


def _two64(e):
    return ((e.to(torch.int64) + 1023) << 52).view(F64)


def _scale64(top, fmt, t):
    """Block scales from the blocks' maxima."""
    if fmt == "nvfp4":
        v = top / 6 / t
        e = torch.where(v > 0, torch.frexp(v).exponent - 1, torch.zeros_like(v, dtype=torch.int32)).clamp(min=-6)
        return torch.minimum(torch.round(v * _two64(3 - e)) * _two64(e - 3), torch.full_like(v, 448))
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, torch.full_like(top, -127, dtype=torch.int32)).clamp(min=-127)
    return _two64(e)


def _held64(v, fmt, t=1.0):
    b = v.reshape(v.shape[0], -1, _block(fmt))
    s = _scale64(b.abs().max(-1).values, fmt, t)[..., None] * t
    mags = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=F64, device=v.device)
    u = torch.where(s > 0, b / s.clamp(min=1e-300), torch.zeros_like(b))
    return (torch.sign(b) * mags[_code64(u)] * s).reshape(v.shape)


def _tensor64(v):
    top = float(v.abs().max())
    return 1.0 if top == 0 else 2.0 ** max(-126, min(127, math.ceil(math.log2(top / 2688))))


def _expert64(w, e, fmt):
    """Expert e's weights [N, K], read from the codes and the scale bytes as they are stored."""
    q = w["q"][e].long()
    N, K = q.shape[0], 2 * q.shape[1]
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=F64, device=q.device)
    v = torch.stack([table[q & 15], table[q >> 4]], dim=2).reshape(N, K)
    n = torch.arange(N, device=q.device)[:, None]
    b = torch.arange(K // _block(fmt), device=q.device)[None]
    chunks = -(-(K // _block(fmt)) // 4)
    at = ((e * N // 128 + e + n // 128) * chunks + b // 4) * 512 + n % 32 * 16 + n % 128 // 32 * 4 + b % 4
    byte = w["s"][at]
    s = byte.view(E4M3).to(F64) if fmt == "nvfp4" else _two64(byte.to(torch.int64) - 127)
    v = v.reshape(N, -1, _block(fmt)) * s[..., None]
    return v.reshape(N, K) * (1.0 if w["t"] is None else float(w["t"][e]))


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


def _exact_select(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    z = s["logits"].double()
    p = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.softmax(z, 1)
    if c["op"] == "select":
        left = p + (0 if s["bias"] is None else s["bias"].double())
        n = E // c["groups"]
        if c["top_groups"] < c["groups"]:
            by = torch.topk(left.reshape(T, -1, n), c["best"], dim=2).values.sum(2)
            out = torch.ones_like(by, dtype=torch.bool)
            for _ in range(c["top_groups"]):
                best = by.argmax(1, keepdim=True)       # the lowest of equals
                out.scatter_(1, best, False)
                by.scatter_(1, best, -math.inf)
            left = left.masked_fill(out.repeat_interleave(n, dim=1), -math.inf)
        picks = []
        for _ in range(k):
            picks.append((left == left.max(1, keepdim=True).values).to(torch.uint8).argmax(1))
            left = left.scatter(1, picks[-1][:, None], -math.inf)
        idx = torch.stack(picks, 1)
        w = torch.gather(p, 1, idx)
        w = w / w.sum(1, keepdim=True) if c["renorm"] else w
        return {"topk_idx": idx.to(torch.int32), "probs": w * c["scale"]}
    # the gradient of the weights of the chosen experts, by the chain rule from the scores
    idx, dw = s["idx"].long(), s["dprobs"].double() * c["scale"]
    q = torch.gather(p, 1, idx)
    if c["renorm"]:
        tot = q.sum(1, keepdim=True)
        dw = dw / tot - (dw * q).sum(1, keepdim=True) / tot ** 2
    dp = torch.zeros_like(p).scatter_add_(1, idx, dw)
    if c["score"] == "sigmoid":
        return {"dlogits": dp * p * (1 - p)}
    return {"dlogits": p * (dp - (dp * p).sum(1, keepdim=True))}


def exact(case, seed):
    if work(case)["flops"] > 9e12:
        return None
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("select"):
        return _exact_select(s)
    fmt = case["fmt"]
    if op == "pack":
        t = 1.0 if s["t"] is None else float(s["t"])
        v = torch.empty((case["T"], case["d"]), dtype=F64, device=DEV)
        v[:] = _held64(s["x"].double(), fmt, t)
        return {"values": v[(s["pair_of_row"] // case["k"]).long()]}
    if op == "pack_w":
        w = s["w"].transpose(1, 2) if case["along"] == "rows" else s["w"]
        return {"values": torch.stack([_held64(x.double().contiguous(), fmt) for x in w])}
    off = s["offsets"].tolist()
    spans = [(e, off[e], off[e + 1]) for e in range(case["E"]) if off[e + 1] > off[e]]
    M = case["M"]
    if op == "mlp":
        x = _held64(s["x"].double(), fmt)
        y = torch.empty((M, case["d"]), dtype=F64, device=DEV)
        for e, a, b in spans:
            h = _held64(_act64(x[a:b] @ _expert64(s["w1"], e, fmt).T, case["act"]), fmt)
            y[a:b] = h @ _expert64(s["w2"], e, fmt).T
        return {"y": y}
    if op == "linear":
        x = _held64(s["a"].double(), fmt)
        z = torch.empty((M, case["N"]), dtype=F64, device=DEV)
        for e, a, b in spans:
            z[a:b] = x[a:b] @ _expert64(s["w"], e, fmt).T
            if s["bias"] is not None:
                z[a:b] += s["bias"][e].double()
        out = _act64(z, case["act"])
        if s["residual"] is not None:
            out = out + s["residual"].double()
        return {"out": out, "z": z} if case["save_z"] else {"out": out}
    g = s["dout"].double()
    g = g if s["z"] is None else _dact64(s["z"].double(), g, case["act"])
    d = g.to(BF).double()
    held = _held64(d, fmt, _tensor64(d) if fmt == "nvfp4" else 1.0)
    da = torch.empty((M, case["K"]), dtype=F64, device=DEV)
    dB = torch.zeros((case["E"], case["K"], case["N"]), dtype=F64, device=DEV)
    db = torch.zeros((case["E"], case["N"]), dtype=F64, device=DEV)
    for e, a, b in spans:
        da[a:b] = held[a:b] @ _expert64(s["w"], e, fmt).T
        dB[e] = s["a"][a:b].double().T @ d[a:b]
        db[e] = g[a:b].sum(0)
    r = {"dz": g, "da": da, "dB": dB}
    if s["bias"] is not None:
        r["dbias"] = db
    return r
