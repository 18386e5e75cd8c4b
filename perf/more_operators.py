"""Cases of the steps between an expert block's products, forward and backward:
pairs sorted by expert with their rows (dispatch), rows brought back to their
tokens with the routing weights (combine) and the gradient of that, the
SiTU-GLU that writes the next product's MXFP8 operand and saves its inputs in
8 bits, its gradient from what was saved, and the RMSNorm's gradient from an
input saved in 8 bits.

A case names its operator ("op") and its sizes.  With `own` false, run()
computes the operator in elementary torch operations in 32 bits; with `own`
true it calls the library.  MXFP8: codes e4m3, blocks of 32 columns share a
power-of-two scale, byte s for 2^(s - 127).
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
TOP = 448.0
SCRATCH = 64 << 20       # bytes of the one workspace that a program keeps for all its calls


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token's latent state to its 16 experts of 896: the smallest call
        {"name": "dispatch_token", "op": "dispatch", "dtype": "mxfp8", "tokens": 1, "topk": 16, "experts": 896, "width": 3584, "pad": 0, "skew": 0.0, "drop": 0.0},
        # a prefill batch of latent states, a tenth of the choices dropped by the router's tail cut
        {"name": "dispatch_prefill", "op": "dispatch", "dtype": "mxfp8", "tokens": 4096, "topk": 16, "experts": 896, "width": 3584, "pad": 0, "skew": 1.0, "drop": 0.1},
        # one token's expert rows back into the hidden state, beside a dense branch
        {"name": "combine_token", "op": "combine", "dtype": "bf16", "out": "bf16", "tokens": 1, "topk": 16, "experts": 896, "width": 7168, "weights": True, "base": True, "drop": 0.0},
        # a prefill batch's fp32 expert rows back into latent states
        {"name": "combine_prefill", "op": "combine", "dtype": "f32", "out": "f32", "tokens": 4096, "topk": 16, "experts": 896, "width": 3584, "weights": True, "base": False, "drop": 0.1},
        # a short batch, few choices, a width that ends inside every vector
        {"name": "combine_grad_odd", "op": "combine_grad", "dtype": "f32", "out": "f32", "tokens": 333, "topk": 6, "experts": 24, "width": 1001, "pad": 0, "drop": 0.2},
        # a training batch: gradients of 65536 expert rows and of their weights
        {"name": "combine_grad_prefill", "op": "combine_grad", "dtype": "bf16", "out": "bf16", "tokens": 4096, "topk": 16, "experts": 896, "width": 3584, "pad": 0, "drop": 0.0},
        # one token's 16 expert rows between gate/up and down, nothing saved
        {"name": "situ_token", "op": "situ", "dtype": "f32", "rows": 16, "inter": 2048, "pad": 0, "save": False},
        # a training batch's rows, gate and up saved in 8 bits
        {"name": "situ_train", "op": "situ", "dtype": "bf16", "rows": 65536, "inter": 2048, "pad": 0, "save": True},
        # ragged rows and an odd number of blocks, fp32 gradients
        {"name": "situ_grad_odd", "op": "situ_grad", "dtype": "f32", "rows": 777, "inter": 1056, "pad": 0},
        # the training batch's gradients
        {"name": "situ_grad_train", "op": "situ_grad", "dtype": "bf16", "rows": 65536, "inter": 2048, "pad": 0},
        # a small batch's hidden states, fp32 gradients, with the residual stream's
        {"name": "norm_grad_batch", "op": "norm_grad", "dtype": "f32", "rows": 64, "width": 7168, "pad": 0, "residual": True},
        # a training batch's hidden states
        {"name": "norm_grad_train", "op": "norm_grad", "dtype": "bf16", "rows": 4096, "width": 7168, "pad": 0, "residual": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("dispatch", "combine", "combine_grad", "situ", "situ_grad", "norm_grad"))
    types = ("f32", "bf16")
    pad = rng.choice((0, 0, 16, 33))
    while True:
        if op in ("dispatch", "combine", "combine_grad"):
            k = rng.randint(1, 16)
            c = {"op": op, "tokens": _log(rng, 1, 8192), "topk": k, "experts": _log(rng, k, 1024), "drop": rng.choice((0.0, 0.0, 0.1, 0.5))}
            if op == "dispatch":
                c.update(dtype=rng.choice(types + ("mxfp8", "mxfp8")), skew=rng.choice((0.0, 0.5, 1.0, 2.0)), pad=pad)
            else:
                c.update(dtype=rng.choice(types), out=rng.choice(types))
            if op == "combine":
                c.update(weights=rng.random() < 0.7, base=rng.random() < 0.5)
            elif op == "combine_grad":
                c.update(pad=pad)
            # widths in whole blocks, in whole vectors, and any
            c["width"] = 32 * _log(rng, 1, 224) if c["dtype"] == "mxfp8" or rng.random() < 0.5 else _log(rng, 8, 7168)
            if c["tokens"] * k * c["width"] * (4 if c["dtype"] == "f32" else 2) <= 65536 * 3584 * 4:
                return c
        elif op in ("situ", "situ_grad"):
            c = {"op": op, "dtype": rng.choice(types), "rows": _log(rng, 1, 65536), "inter": 32 * _log(rng, 1, 128), "pad": 8 * rng.choice((0, 0, 1, 5))}
            if op == "situ":
                c["save"] = rng.random() < 0.7
            if c["rows"] * c["inter"] * (2 if c["dtype"] == "f32" else 1) <= 65536 * 2048:
                return c
        else:
            c = {"op": op, "dtype": rng.choice(types), "rows": _log(rng, 1, 8192), "width": 32 * _log(rng, 2, 512),
                 "pad": 8 * rng.choice((0, 0, 1, 5)), "residual": rng.random() < 0.7}
            if c["rows"] * c["width"] <= 4096 * 7168:
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


def _grads(rows, cols, g):
    """Gradients: normals around 2^-10, rows of uneven size."""
    s = torch.exp(torch.randn(rows, 1, generator=g, device=DEV)) * 2.0 ** -10
    return torch.randn(rows, cols, generator=g, device=DEV) * s


def _wide(x, dtype, pad):
    """The rows of x in a buffer whose rows are `pad` elements longer."""
    wide = torch.zeros(x.shape[0], x.shape[1] + pad, dtype=dtype, device=DEV)
    wide[:, :x.shape[1]] = x.to(dtype)
    return wide[:, :x.shape[1]]


def _mxfp8(x):
    """Codes and scale bytes of what an earlier call quantised."""
    r, c = x.shape
    b = x.view(r, c // 32, 32)
    e = torch.ceil(torch.log2(b.abs().amax(-1).double() / TOP)).clamp(-127, 127)
    q = (b / torch.exp2(e).float()[..., None]).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).reshape(r, c), (e + 127).to(torch.uint8)


def _choices(case, g):
    """Experts of each token as a router picks them (distinct, dropped ones -1) and their weights."""
    t, k, n = case["tokens"], case["topk"], case["experts"]
    u = torch.rand(t, n, generator=g, device=DEV).clamp(1e-6, 1.0 - 1e-6)
    logits = case.get("skew", 0.5) * torch.randn(n, generator=g, device=DEV) - torch.log(-torch.log(u))
    score, idx = torch.sigmoid(logits - 4.0).topk(k, dim=1)
    gone = torch.rand(t, k, generator=g, device=DEV) < case["drop"]
    score = torch.where(gone, torch.zeros_like(score), score)
    w = score / score.sum(1, keepdim=True).clamp(min=1e-9)
    return torch.where(gone, torch.full_like(idx, -1), idx).to(torch.int32), w.contiguous()


def _sorted(idx, n):
    """offsets, perm and place of pairs [T, K] in the order of their experts."""
    flat = idx.reshape(-1)
    key, order = torch.sort(torch.where(flat < 0, torch.full_like(flat, n), flat), stable=True)
    offsets = torch.searchsorted(key, torch.arange(n + 1, dtype=key.dtype, device=DEV), out_int32=True)
    row = torch.arange(order.numel(), dtype=torch.int32, device=DEV)
    place = torch.empty_like(row)
    place[order] = torch.where(key < n, row, torch.full_like(row, -1))
    perm = torch.where(row < offsets[-1], order.to(torch.int32), torch.zeros_like(row))
    return offsets, perm, place.view(idx.shape)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"op": op}
    if op in ("dispatch", "combine", "combine_grad"):
        t, k, c = case["tokens"], case["topk"], case["width"]
        st["idx"], st["w"] = _choices(case, g)
        i32 = dict(dtype=torch.int32, device=DEV)
        st["offsets"], st["perm"], st["place"] = torch.zeros(case["experts"] + 1, **i32), torch.zeros(t * k, **i32), torch.zeros(t, k, **i32)
        if op == "dispatch":
            st["scales"] = st["xs"] = None
            if case["dtype"] == "mxfp8":
                codes, st["xs"] = _mxfp8(_states(t, c, g))
                st["x"] = _wide(codes, torch.uint8, 16 * (case["pad"] // 16))
                st["rows"] = torch.zeros(t * k, c, dtype=torch.uint8, device=DEV)
                st["scales"] = torch.zeros(t * k, c // 32, dtype=torch.uint8, device=DEV)
            else:
                st["x"] = _wide(_states(t, c, g), DTYPES[case["dtype"]], case["pad"])
                st["rows"] = torch.zeros(t * k, c, dtype=DTYPES[case["dtype"]], device=DEV)
            st["workspace"] = torch.empty(SCRATCH, dtype=torch.uint8, device=DEV)
            return st
        st["place"] = _sorted(st["idx"], case["experts"])[2]
        st["rows"] = _states(t * k, c, g).to(DTYPES[case["dtype"]])
        out = DTYPES[case["out"]]
        if op == "combine":
            st["base"] = _states(t, c, g).to(out) if case["base"] else None
            st["y"] = torch.empty(t, c, dtype=out, device=DEV)
            if not case["weights"]:
                st["w"] = None
        else:
            st["dy"] = _wide(_grads(t, c, g), out, case["pad"])
            st["drows"] = torch.zeros_like(st["rows"])
            st["dw"] = torch.empty_like(st["w"])
        return st
    r, dt = case["rows"], DTYPES[case["dtype"]]
    u8 = dict(dtype=torch.uint8, device=DEV)
    if op in ("situ", "situ_grad"):
        f = case["inter"]
        gu = _states(r, 2 * f, g)
        if op == "situ":
            st["gu"] = _wide(gu, dt, case["pad"])
            st["codes"], st["scales"] = torch.empty(r, f, **u8), torch.empty(r, f // 32, **u8)
            st["h"] = torch.empty(r, f, dtype=torch.bfloat16, device=DEV)
            st["saved"] = st["saved_scales"] = None
            if case["save"]:
                st["saved"], st["saved_scales"] = torch.empty(r, 2 * f, **u8), torch.empty(r, 2 * f // 32, **u8)
                st["kept"] = torch.empty(r, 2 * f, dtype=torch.bfloat16, device=DEV)
        else:
            st["saved"], st["saved_scales"] = _mxfp8(gu)
            st["dh"] = _wide(_grads(r, f, g), dt, case["pad"])
            st["dgu"] = torch.empty(r, 2 * f, dtype=dt, device=DEV)
        return st
    c = case["width"]
    st["saved"], st["saved_scales"] = _mxfp8(_states(r, c, g) + 2.0 * torch.randn(r, c, generator=g, device=DEV))
    st["weight"] = (1.0 + 0.1 * torch.randn(c, generator=g, device=DEV)).to(torch.bfloat16)
    st["dn"] = _wide(_grads(r, c, g), dt, case["pad"])
    st["dres"] = _grads(r, c, g).to(dt) if case["residual"] else None
    st["dx"] = torch.empty(r, c, dtype=dt, device=DEV)
    st["dweight"] = torch.empty(c, device=DEV)
    st["workspace"] = torch.empty(SCRATCH, **u8)
    return st


# ------------------------------------------------------------- plain form --

def _quantised(x):
    """The values that the MXFP8 codes of fp32 rows x stand for, in fp32."""
    r, c = x.shape
    b = x.reshape(r, c // 32, 32)
    f, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    e = (e - 9 + (f > 0.875)).clamp(min=-127)
    return torch.ldexp(torch.ldexp(b, -e).to(torch.float8_e4m3fn).float(), e).reshape(r, c)


def _values(codes, scales):
    x = codes.view(torch.float8_e4m3fn).float().reshape(*scales.shape, 32)
    return (x * torch.exp2(scales.float() - 127.0)[..., None]).reshape(codes.shape)


def _gathered(st):
    """fp32 rows of each pair [T, K, W], zeros where the pair was dropped."""
    live = st["place"] >= 0
    return torch.where(live[..., None], st["rows"][st["place"].clamp(min=0).long()].float(), torch.zeros((), device=DEV)), live


def _plain(st):
    op = st["op"]
    if op == "dispatch":
        n = st["offsets"].numel() - 1
        offsets, perm, place = _sorted(st["idx"], n)
        token = torch.div(perm.long(), place.shape[1], rounding_mode="floor")
        live = torch.arange(perm.numel(), device=DEV)[:, None] < offsets[-1]
        move = lambda x: torch.where(live, x[token], torch.zeros((), dtype=x.dtype, device=DEV))
        out = {"offsets": offsets, "perm": perm, "place": place, "rows": move(st["x"])}
        if st["xs"] is not None:
            out["scales"] = move(st["xs"])
        return out
    if op == "combine":
        rows, _ = _gathered(st)
        y = (rows if st["w"] is None else rows * st["w"][..., None]).sum(1)
        if st["base"] is not None:
            y = y + st["base"].float()
        return {"y": y.to(st["y"].dtype)}
    if op == "combine_grad":
        rows, live = _gathered(st)
        dy, n = st["dy"].float(), st["rows"].shape[0]
        drows = torch.zeros(n + 1, dy.shape[1], dtype=st["rows"].dtype, device=DEV)      # dropped pairs' go to the last row
        to = torch.where(live, st["place"], torch.full_like(st["place"], n)).reshape(-1).long()
        drows[to] = (st["w"][..., None] * dy[:, None, :]).to(drows.dtype).flatten(0, 1)
        return {"drows": drows[:n],
                "dw": (rows * dy[:, None, :]).sum(-1)}
    if op == "situ":
        g, u = st["gu"].float().chunk(2, dim=1)
        h = 4.0 * torch.tanh(g / 4.0) / (1.0 + torch.exp(-g)) * 25.0 * torch.tanh(u / 25.0)
        out = {"h": _quantised(h).to(torch.bfloat16)}
        if st["saved"] is not None:
            out["saved"] = _quantised(st["gu"].float()).to(torch.bfloat16)
        return out
    if op == "situ_grad":
        g, u = _values(st["saved"], st["saved_scales"]).chunk(2, dim=1)
        dh = st["dh"].float()
        s, n = 1.0 / (1.0 + torch.exp(-g)), 1.0 / (1.0 + torch.exp(g))
        t, v = torch.tanh(g / 4.0), torch.tanh(u / 25.0)
        dg = dh * 25.0 * v * s * (1.0 / torch.cosh(g / 4.0).square() + 4.0 * t * n)
        du = dh * 4.0 * t * s / torch.cosh(u / 25.0).square()
        return {"dgu": torch.cat([dg, du], 1).to(st["dgu"].dtype)}
    x, dn = _values(st["saved"], st["saved_scales"]), st["dn"].float()
    k = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n, a = x * k, dn * st["weight"].float()
    dx = k * (a - n * (a * n).mean(-1, keepdim=True))
    if st["dres"] is not None:
        dx = dx + st["dres"].float()
    return {"dx": dx.to(st["dx"].dtype), "dweight": (dn * n).sum(0)}


# -------------------------------------------------------------------- run --

def run(state):
    if not own:
        return _plain(state)
    import mxfp4_routed_expert_k3mx_gb300 as k3mx
    st, op = state, state["op"]
    if op == "dispatch":
        k3mx.k3mx_sort(st["offsets"], st["perm"], st["place"], st["idx"], st["workspace"])
        k3mx.k3mx_dispatch(st["rows"], st["x"], st["place"], scales=st["scales"], x_scales=st["xs"])
        out = {"offsets": st["offsets"], "perm": st["perm"], "place": st["place"], "rows": st["rows"]}
        if st["xs"] is not None:
            out["scales"] = st["scales"]
        return out
    if op == "combine":
        k3mx.k3mx_combine(st["y"], st["rows"], st["place"], w=st["w"], base=st["base"])
        return {"y": st["y"]}
    if op == "combine_grad":
        k3mx.k3mx_combine_backward(st["drows"], st["dw"], st["dy"], st["rows"], st["place"], st["w"])
        return {"drows": st["drows"], "dw": st["dw"]}
    if op == "situ":
        k3mx.k3mx_situ_mx(st["codes"], st["scales"], st["gu"], saved=st["saved"], saved_scales=st["saved_scales"])
        k3mx.k3mx_mx_dequantize(st["h"], st["codes"], st["scales"], k3mx.K3MX_MXFP8)
        out = {"h": st["h"]}
        if st["saved"] is not None:
            k3mx.k3mx_mx_dequantize(st["kept"], st["saved"], st["saved_scales"], k3mx.K3MX_MXFP8)
            out["saved"] = st["kept"]
        return out
    if op == "situ_grad":
        k3mx.k3mx_situ_mx_backward(st["dgu"], st["dh"], st["saved"], st["saved_scales"])
        return {"dgu": st["dgu"]}
    k3mx.k3mx_rmsnorm_mx_backward(st["dx"], st["dweight"], st["dn"], st["saved"], st["saved_scales"], st["weight"], EPS,
                                  st["workspace"], dres=st["dres"])
    return {"dx": st["dx"], "dweight": st["dweight"]}


def work(case):
    op = case["op"]
    size = {"f32": 4.0, "bf16": 2.0, "mxfp8": 33.0 / 32.0}
    if op in ("dispatch", "combine", "combine_grad"):
        t, c, p = case["tokens"], case["width"], case["tokens"] * case["topk"]
        live = p * (1.0 - case["drop"])
        e = size[case["dtype"]]
        if op == "dispatch":
            return {"bytes": t * c * e + live * c * e + 4.0 * (2 * p + live + case["experts"] + 1), "flops": 0.0}
        o = size[case["out"]]
        if op == "combine":
            return {"bytes": live * c * e + t * c * o * (2 if case["base"] else 1) + (8.0 if case["weights"] else 4.0) * p, "flops": 2.0 * live * c}
        return {"bytes": 2 * live * c * e + t * c * o + 12.0 * p, "flops": 3.0 * live * c}
    r, s, m = case["rows"], size[case["dtype"]], size["mxfp8"]
    if op == "situ":
        f = case["inter"]
        return {"bytes": r * f * (2 * s + m + 2 + (2 * m + 4 if case["save"] else 0)), "flops": 20.0 * r * f}
    if op == "situ_grad":
        f = case["inter"]
        return {"bytes": r * f * (2 * m + 3 * s), "flops": 30.0 * r * f}
    c = case["width"]
    return {"bytes": r * c * (m + (3 if case["residual"] else 2) * s) + 6.0 * c, "flops": 12.0 * r * c}


# ------------------------------------------------------------------ exact --

def _exact_block(x):
    """Nearest e4m3 values under each block's scale by distance, ties to the even code, rows of doubles."""
    code = torch.arange(127, device=x.device)
    e, m = code // 8, (code % 8).double()
    grid = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10))
    b = x.reshape(-1, 32)
    m = b.abs().amax(1, keepdim=True)
    e = torch.where(m > 0, torch.ceil(torch.log2(m / TOP)), torch.full_like(m, -127.0)).clamp(min=-127.0)
    a = b.abs() / torch.exp2(e)
    hi = torch.searchsorted(grid, a.contiguous()).clamp(1, grid.numel() - 1)
    lo = hi - 1
    dh, dl = grid[hi] - a, a - grid[lo]
    k = torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return (torch.copysign(grid[k], b) * torch.exp2(e)).reshape(x.shape)


def _doubles(codes, scales):
    v = codes.view(torch.float8_e4m3fn).double().reshape(codes.shape[0], -1, 32)
    return (v * (2.0 ** (scales.double() - 127.0))[:, :, None]).reshape(codes.shape)


def _by_rows(rows, cols, f):
    """f(first, last) of runs of rows, its results (tuples of doubles) one below the other."""
    step = max(1, (1 << 24) // cols)
    parts = [f(i, min(i + step, rows)) for i in range(0, rows, step)]
    return [torch.cat(p) for p in zip(*parts)]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "dispatch":
        return None                  # whole numbers, and values that are moved
    if op in ("combine", "combine_grad"):
        place, t, c = st["place"].long(), case["tokens"], case["width"]
        if op == "combine":
            y = torch.zeros(t, c, dtype=torch.float64, device=DEV) if st["base"] is None else st["base"].double()
            for k in range(case["topk"]):
                at = (place[:, k] >= 0).nonzero()[:, 0]
                w = 1.0 if st["w"] is None else st["w"][at, k].double()[:, None]
                y[at] += w * st["rows"][place[at, k]].double()
            return {"y": y}
        drows = torch.zeros(st["rows"].shape, dtype=torch.float64, device=DEV)
        dw = torch.zeros(t, case["topk"], dtype=torch.float64, device=DEV)
        dy = st["dy"].double()
        for k in range(case["topk"]):
            at = (place[:, k] >= 0).nonzero()[:, 0]
            drows[place[at, k]] = st["w"][at, k].double()[:, None] * dy[at]
            dw[at, k] = torch.linalg.vecdot(st["rows"][place[at, k]].double(), dy[at])
        return {"drows": drows, "dw": dw}
    rows = case["rows"]
    if op == "situ":
        f = case["inter"]

        def part(i, j):
            x = st["gu"][i:j].double()
            g, u = x[:, :f], x[:, f:]
            h = _exact_block(100.0 * torch.tanh(0.25 * g) * torch.sigmoid(g) * torch.tanh(0.04 * u))
            return (h, _exact_block(x.contiguous())) if case["save"] else (h,)
        return dict(zip(("h", "saved"), _by_rows(rows, 2 * f, part)))
    if op == "situ_grad":
        f = case["inter"]

        def part(i, j):
            x, dh = _doubles(st["saved"][i:j], st["saved_scales"][i:j]), st["dh"][i:j].double()
            g, u = x[:, :f], x[:, f:]
            t, s, v = torch.tanh(0.25 * g), torch.sigmoid(g), torch.tanh(0.04 * u)
            slope = (1.0 - t) * (1.0 + t) * s + 4.0 * t * s * torch.sigmoid(-g)
            return (torch.cat([25.0 * v * slope * dh, 4.0 * t * s * (1.0 - v) * (1.0 + v) * dh], 1),)
        return {"dgu": _by_rows(rows, 2 * f, part)[0]}
    x, dn, w = _doubles(st["saved"], st["saved_scales"]), st["dn"].double(), st["weight"].double()
    var = x.square().sum(1) / case["width"] + EPS
    a = dn * w
    dot = torch.linalg.vecdot(a, x) / case["width"]
    dx = a / var.sqrt()[:, None] - x * (dot / var.pow(1.5))[:, None]
    if st["dres"] is not None:
        dx = dx + st["dres"].double()
    return {"dx": dx, "dweight": (dn * x / var.sqrt()[:, None]).sum(0)}
