"""Cases of the products with NVFP4 matrices: a linear layer with bias, activation and residual, a gated
pair of projections, and the input gradients of both, for one matrix or for the experts of a layer.

`run` computes a case either in its plain form (elementary torch operations in binary32) or, with
`own` set, through the library's entry points. Both read the same matrices: 4-bit codes
[experts, out, in/2] (two a byte, the even column in the low nibble), one E4M3 scale byte per 16
columns [experts, out, in/16] and a binary32 scale S [experts]. A weight is S * level * E4M3(scale).

The rows of an expert lie back to back, expert e's at offsets[e] .. offsets[e+1] - 1; how many each
has comes from a case's `layout` number alone, the values come from the seed.
"""
import math
import random

import torch

own = False

_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --- the cases ----------------------------------------------------------------------------------

def listed():
    return [
        # one token through an 8B-shaped down projection, onto the residual stream: latency
        _linear("linear_one", tokens=1, out=4096, inp=14336, residual=True),
        # a serving batch's next tokens through a 70B-shaped down projection
        _linear("linear_batch", tokens=64, out=8192, inp=28672, residual=True),
        # a long prompt through an 8B-shaped attention projection with a bias
        _linear("linear_prompt", tokens=8192, out=4096, inp=4096, bias=True),
        # a small classifier-like layer in binary32, nothing a multiple of a tile
        _linear("linear_odd", tokens=333, out=1003, inp=2064, bias=True, act="gelu", dtype="float32"),
        # the down projections of 128 experts, prompts routed unevenly
        _linear("linear_experts", tokens=16384, out=2048, inp=768, experts=128, layout=5),
        # one token through a 70B-shaped gate and up projection
        _gated("gated_one", tokens=1, out=28672, inp=8192),
        # a long prompt through an 8B-shaped gate and up projection
        _gated("gated_prompt", tokens=8192, out=14336, inp=4096),
        # a decode step of 64 requests with 8 of 128 experts each
        _gated("gated_experts", tokens=512, out=768, inp=2048, experts=128, layout=8),
        # adapter training behind a frozen 8B-shaped down projection
        _linear_backward("linear_backward", tokens=4096, out=4096, inp=14336),
        # the small binary32 layer's gradient
        _linear_backward("linear_backward_odd", tokens=333, out=1003, inp=2064, bias=True, act="gelu",
                         dtype="float32"),
        # training through a frozen 8B-shaped gate and up projection
        _gated_backward("gated_backward", tokens=4096, out=14336, inp=4096),
        # training through the frozen experts of a layer
        _gated_backward("gated_backward_experts", tokens=16384, out=768, inp=2048, experts=128,
                        layout=12),
    ]


def _case(op, name, tokens, out, inp, experts=1, act="none", bias=False, residual=False, pre=False,
          dtype="bfloat16", layout=0):
    c = {"op": op, "tokens": tokens, "out": out, "in": inp, "experts": experts, "act": act,
         "bias": bias, "residual": residual, "pre": pre, "dtype": dtype, "layout": layout}
    return dict(c, name=name) if name else c


def _linear(name, **kw):
    return _case("linear", name, **kw)


def _gated(name, act="silu", **kw):
    return _case("gated", name, act=act, **kw)


def _linear_backward(name, **kw):
    return _case("linear_backward", name, **kw)


def _gated_backward(name, act="silu", **kw):
    return _case("gated_backward", name, act=act, **kw)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "gated", "linear_backward", "gated_backward"))
    pairs = 2 if op.startswith("gated") else 1
    experts = 1 if rng.random() < 0.6 else _log(rng, 2, 128)
    out, inp = _log(rng, 16, 28672), 16 * _log(rng, 4, 1792)
    while pairs * experts * out * inp > 2 * 28672 * 8192:
        if experts > 1:
            experts //= 2
        elif out > inp:
            out = out // 2 + 1
        else:
            inp = inp // 32 * 16
    tokens = _log(rng, 1, 16384)
    while pairs * tokens * out * inp > 2 * 8192 * 14336 * 4096 or tokens * (2 * out + inp) > 1 << 29:
        tokens = tokens // 2
    act = rng.choice(("silu", "gelu", "gelu_tanh", "relu"))
    if pairs == 1 and rng.random() < 0.5:
        act = "none"
    linear = op == "linear"
    return _case(op, None, tokens, out, inp, experts, act,
                 bias=pairs == 1 and rng.random() < 0.5, residual=linear and rng.random() < 0.5,
                 pre=not op.endswith("backward") and (act != "none") and rng.random() < 0.3,
                 dtype=rng.choice(("bfloat16", "bfloat16", "bfloat16", "float32")),
                 layout=rng.randrange(1 << 20))


def _counts(c):
    """Rows of each expert: uneven shares, some experts without any."""
    E, T = c["experts"], c["tokens"]
    if E == 1:
        return [T]
    r = random.Random(c["layout"])
    share = [1 / (1 + i) for i in range(E)]
    r.shuffle(share)
    share = [0 if r.random() < 0.05 else s for s in share]
    share[r.randrange(E)] += 0.01
    total, cuts, run = sum(share), [0], 0.0
    for s in share:
        run += s
        cuts.append(min(T, int(round(T * run / total))))
    cuts[-1] = T
    return [b - a for a, b in zip(cuts, cuts[1:])]


# --- what a program has in hand -----------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _e2m1(x):
    """Index of the nearest E2M1 level of x >= 0, ties to the even index, saturating."""
    return ((x > 0.25).to(torch.uint8) + (x >= 0.75) + (x > 1.25) + (x >= 1.75) + (x > 2.5)
            + (x >= 3.5) + (x > 5.0))


def _matrix(g, c):
    """Codes, scale bytes and S of random matrices [experts, out, in], by the max-abs rule."""
    E, out, inp = c["experts"], c["out"], c["in"]
    packed = torch.empty((E, out, inp // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((E, out, inp // 16), dtype=torch.uint8, device="cuda")
    S = 0.02 * (4.5 + torch.rand(E, generator=g, device="cuda")) / (6 * 448)
    rows = max(1, (1 << 26) // inp)
    flat, flat_scales = packed.view(E * out, -1), scales.view(E * out, -1)
    of = S.repeat_interleave(out)
    for at in range(0, E * out, rows):
        n = min(rows, E * out - at)
        w = torch.randn((n, inp // 16, 16), generator=g, device="cuda") * 0.02
        top = w.abs().amax(-1)
        Sr = of[at:at + n, None]
        b = (top / 6 / Sr).clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8).clamp(min=1)
        eff = b.view(torch.float8_e4m3fn).float() * Sr
        i = _e2m1(w.abs() / eff[..., None]) | ((w < 0).to(torch.uint8) << 3)
        i = i.flatten(1)
        flat[at:at + n] = i[:, 0::2] | (i[:, 1::2] << 4)
        flat_scales[at:at + n] = b
    return packed, scales, S


def prepare(case, seed):
    c = dict(case)
    g = _gen(seed)
    T, out, inp, dtype = c["tokens"], c["out"], c["in"], getattr(torch, c["dtype"])
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    counts = _counts(c)
    s = {"case": c, "counts": counts, "W": _matrix(g, c),
         "offsets": torch.tensor([0] + counts).cumsum(0).cuda() if c["experts"] > 1 else None}
    gated = c["op"].startswith("gated")
    if gated:
        s["W2"] = _matrix(g, c)
    if c["op"] in ("linear", "gated"):
        spread = torch.exp(0.7 * randn(inp)) * math.sqrt(512 / inp)       # hot and cold channels
        s["X"] = (randn(T, inp) * spread).to(dtype)
        s["residual"] = randn(T, out).to(dtype) if c["residual"] else None
        s["bias"] = (0.5 * randn(c["experts"], out)).to(dtype) if c["bias"] else None
    else:
        s["dY"] = (0.01 * randn(T, out)).to(dtype)
        if gated:
            s["G"], s["U"] = randn(T, out).to(dtype), randn(T, out).to(dtype)
        elif c["act"] != "none":
            s["Z"] = randn(T, out).to(dtype)
    return s


# --- one pass -----------------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"linear": _run_linear, "gated": _run_gated, "linear_backward": _run_linear_backward,
            "gated_backward": _run_gated_backward}[s["case"]["op"]](s)


def _handles(s):
    """The library's handles of the matrices, made once as a program would."""
    if "nv" not in s:
        from block_scale_search_amd import nvfp4
        s["M"] = nvfp4.Matrix(*s["W"])
        if "W2" in s:
            s["M2"] = nvfp4.Matrix(*s["W2"])
        s["act"] = {"none": nvfp4.ACT_NONE, "silu": nvfp4.ACT_SILU, "gelu": nvfp4.ACT_GELU,
                    "gelu_tanh": nvfp4.ACT_GELU_TANH, "relu": nvfp4.ACT_RELU}[s["case"]["act"]]
        s["nv"] = nvfp4
    return s["nv"], s["act"]


def _run_own(s):
    c = s["case"]
    nv, act = _handles(s)
    if c["op"] == "linear":
        r = nv.linear(s["M"], s["X"], bias=s["bias"], activation=act, residual=s["residual"],
                      seg_offsets=s["offsets"], with_pre=c["pre"])
        return {"Y": r[0], "Z": r[1]} if c["pre"] else {"Y": r}
    if c["op"] == "gated":
        r = nv.gated(s["M"], s["M2"], s["X"], activation=act, seg_offsets=s["offsets"],
                     with_pre=c["pre"])
        return {"H": r[0], "G": r[1], "U": r[2]} if c["pre"] else {"H": r}
    if c["op"] == "linear_backward":
        r = nv.linear_backward(s["M"], s["dY"], Z=s.get("Z"), activation=act,
                               seg_offsets=s["offsets"], with_bias=c["bias"])
        return {k: r[k] for k in ("dX", "dZ", "dbias") if r[k] is not None}
    r = nv.gated_backward(s["M"], s["M2"], s["dY"], s["G"], s["U"], activation=act,
                          seg_offsets=s["offsets"])
    return {k: r[k] for k in ("dX", "dG", "dU")}


def _weights(W, e):
    """Expert e's weights over S, [out, in] binary32 (exact)."""
    packed, scales, _ = W
    lev = torch.tensor(_LEVELS + tuple(-v for v in _LEVELS), device="cuda")
    v = torch.stack([lev[(packed[e] & 15).int()], lev[(packed[e] >> 4).int()]], -1).flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * scales[e].view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _forward_product(s, W):
    """[tokens, out] binary32: X times its expert's transposed weights."""
    x, parts, at = s["X"].float(), [], 0
    for e, n in enumerate(s["counts"]):
        if n:
            parts.append((x[at:at + n] @ _weights(W, e).t()) * W[2][e])
        at += n
    return torch.cat(parts)


def _backward_product(s, W, d):
    """[tokens, in] binary32: d times its expert's weights."""
    parts, at = [], 0
    for e, n in enumerate(s["counts"]):
        if n:
            parts.append((d[at:at + n] @ _weights(W, e)) * W[2][e])
        at += n
    return torch.cat(parts)


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, 0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)


def _expert_of_row(s):
    n = torch.tensor(s["counts"], device="cuda")
    return torch.repeat_interleave(torch.arange(len(n), device="cuda"), n)


def _run_linear(s):
    c, dtype = s["case"], s["X"].dtype
    z = _forward_product(s, s["W"])
    if s["bias"] is not None:
        z = z + s["bias"].float()[_expert_of_row(s)]
    y = _act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"Y": y.to(dtype), "Z": z.to(dtype)} if c["pre"] else {"Y": y.to(dtype)}


def _run_gated(s):
    c, dtype = s["case"], s["X"].dtype
    g, u = _forward_product(s, s["W"]), _forward_product(s, s["W2"])
    h = (_act(g, c["act"]) * u).to(dtype)
    return {"H": h, "G": g.to(dtype), "U": u.to(dtype)} if c["pre"] else {"H": h}


def _run_linear_backward(s):
    c, dtype = s["case"], s["dY"].dtype
    d, r = s["dY"].float(), {}
    if c["act"] != "none":
        d = d * _act_slope(s["Z"].float(), c["act"])
        r["dZ"] = d.to(dtype)
    r["dX"] = _backward_product(s, s["W"], d).to(dtype)
    if c["bias"]:
        r["dbias"] = torch.stack([x.sum(0) for x in d.split(s["counts"])])
    return r


def _run_gated_backward(s):
    c, dtype = s["case"], s["dY"].dtype
    d, g, u = s["dY"].float(), s["G"].float(), s["U"].float()
    dg, du = d * u * _act_slope(g, c["act"]), d * _act(g, c["act"])
    dx = _backward_product(s, s["W"], dg) + _backward_product(s, s["W2"], du)
    return {"dX": dx.to(dtype), "dG": dg.to(dtype), "dU": du.to(dtype)}


# --- what a pass cannot do without --------------------------------------------------------------

def work(case):
    c = case
    size = 2 if c["dtype"] == "bfloat16" else 4
    T, out, inp = c["tokens"], c["out"], c["in"]
    matrices = (2 if c["op"].startswith("gated") else 1)
    used = sum(n > 0 for n in _counts(c))
    wide, bias = T * out * size, c["experts"] * out * size if c["bias"] else 0
    moved = T * inp * size + matrices * used * out * inp * 9 // 16
    if c["op"] == "linear":
        moved += wide * (1 + c["residual"] + c["pre"]) + bias
    elif c["op"] == "gated":
        moved += wide * (1 + 2 * c["pre"])
    elif c["op"] == "linear_backward":
        moved += wide * (1 if c["act"] == "none" else 3) + (c["experts"] * out * 4 if c["bias"] else 0)
    else:
        moved += wide * 5
    return {"bytes": moved, "flops": 2 * matrices * T * out * inp}


# --- the definition in 64 bits ------------------------------------------------------------------

def _exact_weights(W, e):
    """Expert e's weights [out, in], from the codes' bit fields."""
    packed, scales, S = (t[e] for t in W)
    code = torch.empty((packed.shape[0], 2 * packed.shape[1]), dtype=torch.uint8, device="cuda")
    code[:, 0::2], code[:, 1::2] = packed % 16, packed // 16
    half = code % 2                                              # mantissa bit
    expo = (code // 2) % 4
    level = torch.where(expo == 0, half.double() / 2, (2 + half).double() * torch.exp2(expo.double() - 2))
    del expo, half
    level = torch.where(code >= 8, -level, level)
    m, x = (scales % 8).double(), (scales // 8).double()
    scale = torch.where(x == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(x - 10))
    return level.mul_((scale * S.double()).repeat_interleave(16, 1))


def _exact_act(z, act):
    """act(z) and its slope in 64 bits."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    # 0.5 (1 + tanh v) is sigmoid(2 v)
    k = 2 * math.sqrt(2 / math.pi)
    p = torch.sigmoid(k * z * (1 + 0.044715 * z ** 2))
    return z * p, p + z * p * (1 - p) * k * (1 + 3 * 0.044715 * z ** 2)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    T, out, inp, f64 = c["tokens"], c["out"], c["in"], torch.float64
    new = lambda n: torch.empty((T, n), dtype=f64, device="cuda")  # noqa: E731
    at = [0]
    for n in s["counts"]:
        at.append(at[-1] + n)
    spans = [(e, slice(at[e], at[e + 1])) for e in range(c["experts"]) if at[e + 1] > at[e]]
    if c["op"] == "linear":
        z = new(out)
        for e, r in spans:
            z[r] = s["X"][r].double() @ _exact_weights(s["W"], e).t().contiguous()
            if s["bias"] is not None:
                z[r] += s["bias"][e].double()
        y = _exact_act(z, c["act"])[0]
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return {"Y": y, "Z": z} if c["pre"] else {"Y": y}
    if c["op"] == "gated":
        g, u = new(out), new(out)
        for e, r in spans:
            x = s["X"][r].double()
            g[r] = x @ _exact_weights(s["W"], e).t().contiguous()
            u[r] = x @ _exact_weights(s["W2"], e).t().contiguous()
        h = _exact_act(g, c["act"])[0] * u
        return {"H": h, "G": g, "U": u} if c["pre"] else {"H": h}
    dx, d = new(inp), s["dY"].double()
    if c["op"] == "linear_backward":
        if c["act"] != "none":
            d = d * _exact_act(s["Z"].double(), c["act"])[1]
        bias = torch.zeros((c["experts"], out), dtype=f64, device="cuda")
        for e, r in spans:
            dx[r] = d[r] @ _exact_weights(s["W"], e)
            bias[e] = d[r].sum(0)
        result = {"dX": dx}
        if c["act"] != "none":
            result["dZ"] = d
        if c["bias"]:
            result["dbias"] = bias
        return result
    a, slope = _exact_act(s["G"].double(), c["act"])
    dg, du = d * s["U"].double() * slope, d * a
    for e, r in spans:
        dx[r] = dg[r] @ _exact_weights(s["W"], e) + du[r] @ _exact_weights(s["W2"], e)
    return {"dX": dx, "dG": dg, "dU": du}
