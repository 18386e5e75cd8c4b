"""A mixture-of-experts block of any expert width on the microscaled
operators, end to end from bf16 masters:

    python examples/moe_block_mx.py [tokens]

quantises the expert weights to MXFP4 once, then per step

  sum, codes = rmsnorm(x + residual)        k3mx_rmsnorm_mx (bf16 copy for the router)
  idx, w     = router(normed)               k3mx_router
  offsets    = grouping of the pairs        k3mx_group
  g | u      = W13[e] x per pair            k3mx_mx_grouped
  h          = SiTU-GLU(g, u) in MXFP8      k3mx_mx_quantize
  rows       = W2[e] h per pair             k3mx_mx_grouped
  y          = sum_k w_k rows + Ws x        k3mx_mx_linear (a dense branch beside the experts)

The router's shapes (hidden 7168, 896 experts, top 16) are the library's; the
experts' and the dense branch's widths are free.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_routed_expert_k3mx_gb300 as k3mx  # noqa: E402

HIDDEN, EXPERTS, TOPK = 7168, k3mx.K3MX_N_EXPERTS, k3mx.K3MX_TOPK
EPS = 1e-5


def u8(*shape):
    return torch.empty(*shape, dtype=torch.uint8, device="cuda")


def quantized(w, fmt):
    """(codes, scales) of a matrix [rows, cols]."""
    rows, cols = w.shape
    codes = u8(rows, cols // 2 if fmt == k3mx.K3MX_MXFP4 else cols)
    return k3mx.k3mx_mx_quantize(codes, u8(rows, cols // 32), w, fmt)


def stacked(n, rows, cols, gen):
    """MXFP4 weights of n matrices [rows, cols], made one master at a time."""
    packed, scales = u8(n, rows, cols // 2), u8(n, rows, cols // 32)
    for i in range(n):
        master = torch.randn(rows, cols, generator=gen, device="cuda", dtype=torch.float32) / cols ** 0.5
        k3mx.k3mx_mx_quantize(packed[i], scales[i], master.bfloat16(), k3mx.K3MX_MXFP4)
    return packed, scales


class Block:
    def __init__(self, inter=256, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.inter = inter
        self.norm = (1 + 0.1 * torch.randn(HIDDEN, generator=gen, device="cuda")).bfloat16()
        self.router = (torch.randn(EXPERTS, HIDDEN, generator=gen, device="cuda") / HIDDEN ** 0.5).bfloat16()
        self.bias = torch.zeros(EXPERTS, device="cuda")
        self.w13 = stacked(EXPERTS, 2 * inter, HIDDEN, gen)
        self.w2 = stacked(EXPERTS, HIDDEN, inter, gen)
        self.dense = tuple(t[0] for t in stacked(1, HIDDEN, HIDDEN, gen))

    def step(self, x, residual):
        """x, residual [T, 7168] bf16 -> every stage's result by name."""
        T, P = x.shape[0], x.shape[0] * TOPK
        bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
        i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")
        r = {"sum": bf(T, HIDDEN), "normed": bf(T, HIDDEN), "codes": u8(T, HIDDEN), "scales": u8(T, HIDDEN // 32)}
        k3mx.k3mx_rmsnorm_mx(r["codes"], r["scales"], r["sum"], x, residual, self.norm, EPS, normed=r["normed"])
        r["logits"], r["idx"], r["w"] = torch.empty(T, EXPERTS, device="cuda"), i32(T, TOPK), torch.empty(T, TOPK, device="cuda")
        k3mx.k3mx_router(r["logits"], r["idx"], r["w"], r["normed"], self.router, self.bias)
        r["offsets"], r["perm"] = i32(EXPERTS + 1), i32(P)
        k3mx.k3mx_group(i32(EXPERTS), r["offsets"], r["perm"], r["idx"], u8(k3mx.k3mx_group_workspace_size(T)))
        r["token"] = r["perm"].long() // TOPK
        xc, xs = r["codes"][r["token"]], r["scales"][r["token"]]
        r["gu"] = torch.empty(P, 2 * self.inter, device="cuda")
        k3mx.k3mx_mx_grouped(r["gu"], xc, xs, *self.w13, r["offsets"])
        g, u = r["gu"].chunk(2, dim=1)
        r["h"] = (4 * torch.tanh(g / 4) * torch.sigmoid(g)) * (25 * torch.tanh(u / 25))
        r["hcodes"], r["hscales"] = quantized(r["h"], k3mx.K3MX_MXFP8)
        r["rows"] = torch.empty(P, HIDDEN, device="cuda")
        k3mx.k3mx_mx_grouped(r["rows"], r["hcodes"], r["hscales"], *self.w2, r["offsets"])
        r["y"] = torch.empty(T, HIDDEN, device="cuda")
        k3mx.k3mx_mx_linear(r["y"], r["codes"], r["scales"], *self.dense)
        r["out"] = r["y"].index_add(0, r["token"], r["rows"] * r["w"].reshape(-1)[r["perm"].long()][:, None])
        return r


def main():
    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 64
    block = Block()
    x = torch.randn(tokens, HIDDEN, device="cuda").bfloat16()
    residual = torch.randn(tokens, HIDDEN, device="cuda").bfloat16()
    block.step(x, residual)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(10):
        out = block.step(x, residual)["out"]
    end.record()
    end.synchronize()
    status, detail = k3mx.k3mx_device_status()
    assert status == 0, (status, detail)
    print(f"{tokens} tokens: {start.elapsed_time(end) / 10:.3f} ms a step, |y| {out.norm().item() / out.numel() ** 0.5:.4f}")


if __name__ == "__main__":
    main()
