"""A step of training through a mixture-of-experts block of any shape whose
expert weights stay frozen in MXFP4: the gradients of its input, its norm's
weight and its router.

    python examples/moe_block_train.py [tokens]

Forward
  sum, codes = rmsnorm(x + residual)        k3mx_rmsnorm_mx; sum saved in 8 bits: k3mx_mx_quantize
  idx, w     = router(normed)               (any router's choices)
  place      = pairs by expert              k3mx_sort
  rows       = the tokens' codes by pair    k3mx_dispatch
  g | u      = W13[e] rows                  k3mx_mx_grouped
  h          = SiTU-GLU(g, u) in MXFP8      k3mx_situ_mx; g | u saved in 8 bits
  out        = W2[e] h                      k3mx_mx_grouped
  y          = sum + sum_k w_k out          k3mx_combine
Backward, from dy
  dout, dw   of the sum over a token's pairs   k3mx_combine_backward
  dh         = dout W2[e]                   (the weights' values, a product an expert)
  dg | du    at the saved g | u             k3mx_situ_mx_backward
  drows      = dg | du W13[e]
  dn         = the pairs' sum by token      k3mx_combine without weights
  dx, dgain  at the saved sum               k3mx_rmsnorm_mx_backward
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_routed_expert_k3mx_gb300 as k3mx  # noqa: E402

EPS = 1e-5


def u8(*shape):
    return torch.empty(*shape, dtype=torch.uint8, device="cuda")


def mxfp8(x):
    return k3mx.k3mx_mx_quantize(u8(*x.shape), u8(x.shape[0], x.shape[1] // 32), x, k3mx.K3MX_MXFP8)


class Block:
    def __init__(self, hidden=512, experts=16, topk=4, inter=256, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")
        self.hidden, self.experts, self.topk, self.inter = hidden, experts, topk, inter
        self.gain = (1 + 0.1 * normal(hidden)).bfloat16()
        self.router = normal(experts, hidden) / hidden ** 0.5
        self.w13, self.w2 = self._frozen(2 * inter, hidden, normal), self._frozen(hidden, inter, normal)

    def _frozen(self, out, cols, normal):
        """(codes, scales, values) of an MXFP4 matrix an expert."""
        packed, scales = u8(self.experts, out, cols // 2), u8(self.experts, out, cols // 32)
        values = torch.empty(self.experts, out, cols, device="cuda")
        for e in range(self.experts):
            k3mx.k3mx_mx_quantize(packed[e], scales[e], 2 * normal(out, cols) / cols ** 0.5, k3mx.K3MX_MXFP4)
            k3mx.k3mx_mx_dequantize(values[e], packed[e], scales[e], k3mx.K3MX_MXFP4)
        return packed, scales, values

    def buffers(self, tokens):
        """What a step of so many tokens writes, once for all steps."""
        T, H, F, K = tokens, self.hidden, self.inter, self.topk
        P = T * K
        f = lambda *s: torch.empty(*s, device="cuda")
        i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")
        workspace = max(k3mx.k3mx_sort_workspace_size(T, K, self.experts), k3mx.k3mx_rmsnorm_mx_backward_workspace_size(T, H))
        return {"codes": u8(T, H), "scales": u8(T, H // 32), "sum": f(T, H), "normed": f(T, H).bfloat16(), "kept": u8(T, H),
                "kept_scales": u8(T, H // 32), "offsets": i32(self.experts + 1), "perm": i32(P), "place": i32(T, K),
                "rows": u8(P, H), "row_scales": u8(P, H // 32), "gu": f(P, 2 * F), "h": u8(P, F), "h_scales": u8(P, F // 32),
                "saved": u8(P, 2 * F), "saved_scales": u8(P, 2 * F // 32), "out": f(P, H), "y": f(T, H), "dout": f(P, H), "dw": f(T, K),
                "dgu": f(P, 2 * F), "dn": f(T, H), "dx": f(T, H), "dgain": f(H), "workspace": u8(workspace)}

    def choices(self, normed):
        """Sigmoid scores, the topk largest, renormalised; (idx, w, scores)."""
        scores = torch.sigmoid(normed.float() @ self.router.T)
        top, idx = scores.topk(self.topk, dim=1)
        return idx.to(torch.int32), top / top.sum(1, keepdim=True), scores

    def forward(self, x, residual, b):
        k3mx.k3mx_rmsnorm_mx(b["codes"], b["scales"], b["sum"], x, residual, self.gain, EPS, normed=b["normed"])
        k3mx.k3mx_mx_quantize(b["kept"], b["kept_scales"], b["sum"], k3mx.K3MX_MXFP8)
        b["idx"], b["w"], b["scores"] = self.choices(b["normed"])
        k3mx.k3mx_sort(b["offsets"], b["perm"], b["place"], b["idx"], b["workspace"])
        k3mx.k3mx_dispatch(b["rows"], b["codes"], b["place"], scales=b["row_scales"], x_scales=b["scales"])
        k3mx.k3mx_mx_grouped(b["gu"], b["rows"], b["row_scales"], *self.w13[:2], b["offsets"])
        k3mx.k3mx_situ_mx(b["h"], b["h_scales"], b["gu"], saved=b["saved"], saved_scales=b["saved_scales"])
        k3mx.k3mx_mx_grouped(b["out"], b["h"], b["h_scales"], *self.w2[:2], b["offsets"])
        return k3mx.k3mx_combine(b["y"], b["out"], b["place"], w=b["w"], base=b["sum"])

    def _through(self, d, weights, b):
        """d W[e] for the rows of each expert (its rows' number is read back: one size a product)."""
        out = torch.empty(d.shape[0], weights.shape[2], device="cuda")
        offsets = b["offsets"].tolist()
        for e in range(self.experts):
            out[offsets[e]:offsets[e + 1]] = d[offsets[e]:offsets[e + 1]] @ weights[e]
        return out

    def backward(self, dy, b):
        """Gradients of the input (x and residual have the same), the norm's
        weight and the router, from that of y."""
        k3mx.k3mx_combine_backward(b["dout"], b["dw"], dy, b["out"], b["place"], b["w"])
        b["dh"] = self._through(b["dout"], self.w2[2], b)
        k3mx.k3mx_situ_mx_backward(b["dgu"], b["dh"], b["saved"], b["saved_scales"])
        b["drows"] = self._through(b["dgu"], self.w13[2], b)
        k3mx.k3mx_combine(b["dn"], b["drows"], b["place"])
        # w = top / sum(top), top = sigmoid(logits) of the chosen
        top = b["scores"].gather(1, b["idx"].long())
        dtop = (b["dw"] - (b["dw"] * b["w"]).sum(1, keepdim=True)) / top.sum(1, keepdim=True)
        b["dlogits"] = torch.zeros_like(b["scores"]).scatter_(1, b["idx"].long(), dtop * top * (1 - top))
        b["drouter"] = b["dlogits"].T @ b["normed"].float()
        b["dn"] += b["dlogits"] @ self.router
        k3mx.k3mx_rmsnorm_mx_backward(b["dx"], b["dgain"], b["dn"], b["kept"], b["kept_scales"], self.gain, EPS, b["workspace"],
                                      dres=dy)
        return b["dx"], b["dgain"], b["drouter"]


def main():
    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 256
    block = Block()
    x, residual, target = (torch.randn(tokens, block.hidden, device="cuda") for _ in range(3))
    b = block.buffers(tokens)
    for step in range(10):
        y = block.forward(x, residual, b)
        loss = (y - target).square().mean()
        dx, dgain, drouter = block.backward(2 * (y - target) / y.numel(), b)
        block.gain = (block.gain.float() - 50 * dgain).bfloat16()
        block.router -= 50 * drouter
        print(f"step {step}: loss {loss.item():.4f}, |dgain| {dgain.norm().item():.3e}, |drouter| {drouter.norm().item():.3e}")
    status, detail = k3mx.k3mx_device_status()
    assert status == 0, (status, detail)


if __name__ == "__main__":
    main()
