"""Cases of the microscaled operators: quantisation, the norm that quantises,
and the dense and the grouped product of MXFP8 activations with MXFP4 weights.

A case names its operator ("op") and its sizes.  With `own` false, run()
computes the operator in elementary torch operations in 32 bits; with `own`
true it calls the library.  Formats (blocks of 32 columns share a power-of-two
scale, byte s for 2^(s - 127)):
  mxfp4  codes e2m1, two per byte, the low nibble the even column
  mxfp8  codes e4m3, one per byte
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token's hidden state before a product: the smallest call
        {"name": "quantize_token", "op": "quantize", "fmt": "mxfp8", "dtype": "bf16", "rows": 1, "cols": 7168, "pad": 0},
        # a prefill batch's states, rows of a wider buffer
        {"name": "quantize_states", "op": "quantize", "fmt": "mxfp8", "dtype": "bf16", "rows": 4096, "cols": 7168, "pad": 512},
        # the gate and up matrices of the fused shared experts, from fp32 masters to the library's weight format
        {"name": "quantize_weights", "op": "quantize", "fmt": "mxfp4", "dtype": "f32", "rows": 12288, "cols": 7168, "pad": 0},
        # one token between two layers, 8-bit output alone
        {"name": "norm_token", "op": "norm", "dtype": "bf16", "rows": 1, "cols": 7168, "normed": False},
        # a prefill batch between two layers, with the bf16 output that a router reads
        {"name": "norm_states", "op": "norm", "dtype": "bf16", "rows": 4096, "cols": 7168, "normed": True},
        # the hidden-to-latent projection of one token
        {"name": "linear_token", "op": "linear", "dtype": "bf16", "rows": 1, "out": 3584, "cols": 7168},
        # a serving batch through the shared experts' gate and up, fp32 output
        {"name": "linear_batch", "op": "linear", "dtype": "f32", "rows": 64, "out": 12288, "cols": 7168},
        # odd sizes: a short prompt, an output that ends inside a tile, few K blocks
        {"name": "linear_odd", "op": "linear", "dtype": "bf16", "rows": 333, "out": 1000, "cols": 1152},
        # a prefill batch through the shared experts' gate and up
        {"name": "linear_prefill", "op": "linear", "dtype": "bf16", "rows": 4096, "out": 12288, "cols": 7168},
        # one token's 16 expert rows over 64 experts
        {"name": "grouped_token", "op": "grouped", "dtype": "bf16", "rows": 16, "groups": 64, "out": 2048, "cols": 3584, "skew": 0.0},
        # ragged groups, some empty, one far larger than the others, odd sizes, fp32 output
        {"name": "grouped_ragged", "op": "grouped", "dtype": "f32", "rows": 777, "groups": 24, "out": 1000, "cols": 1152, "skew": 2.0},
        # a prefill batch's rows over 64 experts' gate and up
        {"name": "grouped_prefill", "op": "grouped", "dtype": "bf16", "rows": 16384, "groups": 64, "out": 4096, "cols": 3584, "skew": 0.5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "norm", "linear", "grouped"))
    dtype = rng.choice(("f32", "bf16"))
    while True:
        if op == "quantize":
            c = {"op": op, "fmt": rng.choice(("mxfp4", "mxfp8")), "dtype": dtype, "rows": _log(rng, 1, 12288),
                 "cols": 32 * _log(rng, 1, 512), "pad": rng.choice((0, 0, 8, 96))}
            if c["rows"] * c["cols"] <= 12288 * 7168:
                return c
        elif op == "norm":
            c = {"op": op, "dtype": dtype, "rows": _log(rng, 1, 8192), "cols": 32 * _log(rng, 2, 512),
                 "normed": rng.random() < 0.5}
            if c["rows"] * c["cols"] <= 8192 * 7168:
                return c
        elif op == "linear":
            c = {"op": op, "dtype": dtype, "rows": _log(rng, 1, 4096), "out": _log(rng, 32, 12288),
                 "cols": 128 * _log(rng, 1, 56)}
            if c["rows"] * c["out"] * c["cols"] <= 4096 * 12288 * 7168:
                return c
        else:
            c = {"op": op, "dtype": dtype, "rows": _log(rng, 1, 16384), "groups": _log(rng, 1, 64),
                 "out": _log(rng, 32, 4096), "cols": 128 * _log(rng, 1, 28), "skew": rng.choice((0.0, 0.5, 1.0, 2.0))}
            if c["rows"] * c["out"] * c["cols"] <= 16384 * 4096 * 3584:
                return c


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _states(rows, cols, g):
    """Activations: unit normals, some channels an order of magnitude larger."""
    ch = torch.exp(0.5 * torch.randn(cols, generator=g, device=DEV))
    ch = torch.where(torch.rand(cols, generator=g, device=DEV) < 0.01, 20.0 * ch, ch)
    return torch.randn(rows, cols, generator=g, device=DEV) * ch


def _mxfp8(x):
    """Codes and scale bytes of activations that an earlier call quantised."""
    r, c = x.shape
    b = x.view(r, c // 32, 32)
    e = torch.ceil(torch.log2(b.abs().amax(-1).double() / 448.0)).clamp(-127, 127)
    q = (b / torch.exp2(e).float()[..., None]).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).reshape(r, c), (e + 127).to(torch.uint8)


def _weights(shape, cols, g):
    """Packed e2m1 codes and scale bytes around 2^-4."""
    p = torch.randint(0, 256, (*shape, cols // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.randint(118, 129, (*shape, cols // 32), generator=g, device=DEV, dtype=torch.uint8)
    return p, s


def prepare(case, seed):
    g = _gen(seed)
    r, c, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
    op = case["op"]
    st = {"op": op, "fmt": case.get("fmt", "mxfp8")}
    if op == "quantize":
        wide = torch.empty(r, c + case["pad"], dtype=dt, device=DEV)
        wide[:, :c] = _states(r, c, g).to(dt)
        st["x"] = wide[:, :c]
    elif op == "norm":
        st["x"] = _states(r, c, g).to(dt)
        st["residual"] = (4.0 * torch.randn(r, c, generator=g, device=DEV)).to(dt)
        st["weight"] = (1.0 + 0.1 * torch.randn(c, generator=g, device=DEV)).to(torch.bfloat16)
        st["sum"] = torch.empty(r, c, dtype=dt, device=DEV)
        st["normed"] = torch.empty(r, c, dtype=torch.bfloat16, device=DEV) if case["normed"] else None
    if op in ("quantize", "norm"):
        st["codes"] = torch.empty(r, c // 2 if st["fmt"] == "mxfp4" else c, dtype=torch.uint8, device=DEV)
        st["scales"] = torch.empty(r, c // 32, dtype=torch.uint8, device=DEV)
        st["values"] = torch.empty(r, c, dtype=dt if op == "quantize" else torch.bfloat16, device=DEV)
        return st
    st["codes"], st["scales"] = _mxfp8(_states(r, c, g))
    st["y"] = torch.empty(r, case["out"], dtype=dt, device=DEV)
    if op == "linear":
        st["packed"], st["wscales"] = _weights((case["out"],), c, g)
        return st
    n = case["groups"]
    st["packed"], st["wscales"] = _weights((n, case["out"]), c, g)
    # rows of a group: a token's choice of experts, from even (skew 0) to a few experts taking most
    p = torch.softmax(case["skew"] * torch.randn(n, generator=g, device=DEV), 0)
    pick = torch.multinomial(p, r, replacement=True, generator=g)
    counts = torch.bincount(pick, minlength=n)
    st["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    st["largest"] = int(counts.max())
    return st


# ------------------------------------------------------------- plain form --

def _quantised(x, fmt):
    """The values that the codes of fp32 rows x stand for, in fp32."""
    r, c = x.shape
    b = x.reshape(r, c // 32, 32)
    f, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    e = (e - 3 + (f > 0.75) if fmt == "mxfp4" else e - 9 + (f > 0.875)).clamp(min=-127)
    a = torch.ldexp(b, -e)
    if fmt == "mxfp4":
        m = a.abs()
        k = (m > 0.25).int() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
        q = torch.tensor(E2M1, device=x.device)[k] * torch.sign(a)
    else:
        q = a.to(torch.float8_e4m3fn).float()
    return torch.ldexp(q, e).reshape(r, c)


def _plain_weight(p, s):
    """fp32 values of packed codes [..., K/2] with scale bytes [..., K/32]."""
    t = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=p.device)
    w = t[torch.stack([p & 15, p >> 4], -1).int()].reshape(*s.shape, 32)
    k = torch.exp2(s.float() - 127.0) * (s != 255)
    return (w * k[..., None]).reshape(*p.shape[:-1], 2 * p.shape[-1])


def _plain_states(c, s):
    x = c.view(torch.float8_e4m3fn).float().reshape(*s.shape, 32)
    return (x * torch.exp2(s.float() - 127.0)[..., None]).reshape(c.shape)


def _plain(st):
    op = st["op"]
    if op == "quantize":
        return {"values": _quantised(st["x"].float(), st["fmt"]).to(st["values"].dtype)}
    if op == "norm":
        s = st["x"].float() + st["residual"].float()
        n = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS) * st["weight"].float()
        out = {"sum": s.to(st["sum"].dtype), "values": _quantised(n, "mxfp8").to(torch.bfloat16)}
        if st["normed"] is not None:
            out["normed"] = n.to(torch.bfloat16)
        return out
    x = _plain_states(st["codes"], st["scales"])
    if op == "linear":
        return {"y": (x @ _plain_weight(st["packed"], st["wscales"]).T).to(st["y"].dtype)}
    off = st["offsets"].long()
    r, n = x.shape[0], off.numel() - 1
    row = torch.arange(r, device=x.device)
    grp = torch.searchsorted(off, row, right=True) - 1
    if r <= n:        # few rows: each with its group's weights
        w = _plain_weight(st["packed"][grp], st["wscales"][grp])
        return {"y": torch.bmm(w, x[:, :, None])[:, :, 0].to(st["y"].dtype)}
    place = row - off[grp]
    box = x.new_zeros(n, st["largest"], x.shape[1])
    box[grp, place] = x
    y = torch.bmm(box, _plain_weight(st["packed"], st["wscales"]).transpose(1, 2))
    return {"y": y[grp, place].to(st["y"].dtype)}


# -------------------------------------------------------------------- run --

def run(state):
    if not own:
        return _plain(state)
    import mxfp4_routed_expert_k3mx_gb300 as k3mx
    op = state["op"]
    fmt = k3mx.K3MX_MXFP4 if state["fmt"] == "mxfp4" else k3mx.K3MX_MXFP8
    if op == "quantize":
        k3mx.k3mx_mx_quantize(state["codes"], state["scales"], state["x"], fmt)
        k3mx.k3mx_mx_dequantize(state["values"], state["codes"], state["scales"], fmt)
        return {"values": state["values"]}
    if op == "norm":
        k3mx.k3mx_rmsnorm_mx(state["codes"], state["scales"], state["sum"], state["x"], state["residual"],
                             state["weight"], EPS, normed=state["normed"])
        k3mx.k3mx_mx_dequantize(state["values"], state["codes"], state["scales"], fmt)
        out = {"sum": state["sum"], "values": state["values"]}
        if state["normed"] is not None:
            out["normed"] = state["normed"]
        return out
    if op == "linear":
        k3mx.k3mx_mx_linear(state["y"], state["codes"], state["scales"], state["packed"], state["wscales"])
    else:
        k3mx.k3mx_mx_grouped(state["y"], state["codes"], state["scales"], state["packed"], state["wscales"],
                             state["offsets"])
    return {"y": state["y"]}


def work(case):
    r, c = case["rows"], case["cols"]
    size = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op == "quantize":
        code = 0.5 if case["fmt"] == "mxfp4" else 1.0
        return {"bytes": r * c * (2 * size + code + 1 / 32), "flops": 3.0 * r * c}
    if op == "norm":
        return {"bytes": r * c * (3 * size + 1 + 1 / 32 + 2 + (2 if case["normed"] else 0)) + 2 * c, "flops": 8.0 * r * c}
    n = case["out"]
    # of the groups, those that hold a row (the expected number, were they even)
    groups = case.get("groups", 1)
    full = groups * (1.0 - (1.0 - 1.0 / groups) ** r)
    return {"bytes": r * c * 33 / 32 + full * n * c * 17 / 32 + r * n * size, "flops": 2.0 * r * n * c}


# ------------------------------------------------------------------ exact --

def _exact_block(x, fmt):
    """Nearest values by distance, ties to the even code, rows of doubles."""
    r, c = x.shape
    if fmt == "mxfp4":
        grid, top = torch.tensor(E2M1, dtype=torch.float64, device=x.device), 6.0
    else:
        code = torch.arange(127, device=x.device)
        e, m = code // 8, (code % 8).double()
        grid, top = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10)), 448.0
    b = x.reshape(-1, 32)
    m = b.abs().amax(1, keepdim=True)
    e = torch.where(m > 0, torch.ceil(torch.log2(m / top)), torch.full_like(m, -127.0)).clamp(min=-127.0)
    a = b.abs() / torch.exp2(e)
    hi = torch.searchsorted(grid, a.contiguous()).clamp(1, grid.numel() - 1)
    lo = hi - 1
    dh, dl = grid[hi] - a, a - grid[lo]
    k = torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return (torch.copysign(grid[k], b) * torch.exp2(e)).reshape(r, c)


def _exact_quantised(x, fmt):
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    step = max(1, (1 << 24) // x.shape[1])
    for i in range(0, x.shape[0], step):
        out[i:i + step] = _exact_block(x[i:i + step].double(), fmt)
    return out


def _exact_weight(p, s):
    w = torch.empty(p.shape[0], p.shape[1], 2, dtype=torch.float64, device=p.device)
    for half, nib in ((0, p % 16), (1, p // 16)):
        mag, odd = (nib % 8) // 2, (nib % 2).double()
        v = torch.where(mag == 0, 0.5 * odd, (1.0 + 0.5 * odd) * 2.0 ** (mag.double() - 1.0))
        w[:, :, half] = torch.where(nib >= 8, -v, v)
    k = torch.where(s == 255, torch.zeros_like(s, dtype=torch.float64), 2.0 ** (s.double() - 127.0))
    return (w.reshape(s.shape[0], -1, 32) * k[:, :, None]).reshape(s.shape[0], -1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return {"values": _exact_quantised(st["x"], st["fmt"])}
    if op == "norm":
        s = st["x"].double() + st["residual"].double()
        n = s / torch.sqrt(s.square().sum(1, keepdim=True) / s.shape[1] + EPS) * st["weight"].double()
        out = {"sum": s, "values": _exact_quantised(n, "mxfp8")}
        if case["normed"]:
            out["normed"] = n
        return out
    x = st["codes"].view(torch.float8_e4m3fn).double()
    x = (x.reshape(x.shape[0], -1, 32) * 2.0 ** (st["scales"].double() - 127.0)[:, :, None]).reshape(x.shape)
    if op == "linear":
        return {"y": x @ _exact_weight(st["packed"], st["wscales"]).T}
    y = torch.empty(case["rows"], case["out"], dtype=torch.float64, device=DEV)
    off = st["offsets"].tolist()
    for i in range(case["groups"]):
        if off[i + 1] > off[i]:
            y[off[i]:off[i + 1]] = x[off[i]:off[i + 1]] @ _exact_weight(st["packed"][i], st["wscales"][i]).T
    return {"y": y}
