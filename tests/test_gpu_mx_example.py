"""The example block's stages, each against the definition applied to what
the stage before wrote (double precision on sampled rows)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import mx_ref
import mxfp4_routed_expert_k3mx_gb300 as k3mx

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block_mx.py")


@pytest.fixture(scope="module")
def example(cuda_dev):
    spec = importlib.util.spec_from_file_location("moe_block_mx", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m, m.Block(inter=128, seed=3)


@pytest.mark.parametrize("tokens", [1, 37])
def test_block_stages(example, tokens):
    m, block = example
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    x, res = (torch.randn(tokens, m.HIDDEN, generator=gen, device="cuda").bfloat16() for _ in range(2))
    r = {k: v.cpu().numpy() if v.dtype != torch.bfloat16 else v.float().cpu().numpy() for k, v in block.step(x, res).items()}
    assert k3mx.k3mx_device_status() == (0, 0)
    # grouping: every pair once, under its expert
    assert r["offsets"][-1] == tokens * m.TOPK and sorted(r["perm"]) == list(range(tokens * m.TOPK))
    expert = np.searchsorted(r["offsets"], np.arange(tokens * m.TOPK), side="right") - 1
    assert np.array_equal(expert, r["idx"].reshape(-1)[r["perm"]])
    pick = np.random.default_rng(0).permutation(tokens * m.TOPK)[:40]
    for p in pick:
        t, e = r["perm"][p] // m.TOPK, expert[p]
        w13, s13, w2, s2 = (v[e].cpu().numpy() for v in (*block.w13, *block.w2))
        y, ad = mx_ref.product(r["codes"][t:t + 1], r["scales"][t:t + 1], w13, s13)
        assert np.all(np.abs(r["gu"][p] - y[0]) <= 1e-5 * ad[0])
        y, ad = mx_ref.product(r["hcodes"][p:p + 1], r["hscales"][p:p + 1], w2, s2)
        assert np.all(np.abs(r["rows"][p] - y[0]) <= 1e-5 * ad[0])
    code, s = mx_ref.quantize(r["h"].astype(np.float64), mx_ref.MXFP8)
    assert np.array_equal(code, r["hcodes"]) and np.array_equal(s, r["hscales"])
    y, ad = mx_ref.product(r["codes"], r["scales"], *(t.cpu().numpy() for t in block.dense))
    assert np.all(np.abs(r["y"] - y) <= 1e-5 * ad)
    # the whole against the routed sum in double (16 fp32 additions a value)
    out = r["y"].astype(np.float64)
    mag = np.abs(out)
    for p in range(tokens * m.TOPK):
        t, k = divmod(int(r["perm"][p]), m.TOPK)
        out[t] += np.float64(r["w"][t, k]) * r["rows"][p]
        mag[t] += np.abs(np.float64(r["w"][t, k]) * r["rows"][p])
    assert np.all(np.abs(r["out"] - out) <= 20 * 2.0 ** -24 * mag)
