"""The microscaled operators without a GPU: the double-precision definitions
pinned by hand, exported symbols, and the refusals of the C ABI and of the
binding."""
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import mx_ref
import mxfp4_routed_expert_k3mx_gb300 as k3mx

FAKE = 0x10000
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "k3mx_mx.h")


def test_definition_by_hand():
    assert mx_ref.E4M3[126] == 448.0 and mx_ref.E4M3[8] == 2.0 ** -6 and mx_ref.E4M3[1] == 2.0 ** -9
    x = np.zeros((1, 96))
    x[0, :4] = 6.0, 5.0, -0.25, 0.75        # ties: 5 -> 4 (even), .25 -> 0, .75 -> 1
    x[0, 32] = 6.0 + 2.0 ** -20             # just above the top: the next scale
    code, s = mx_ref.quantize(x, mx_ref.MXFP4)
    assert list(s[0]) == [127, 128, 0]
    assert list(code[0, :4]) == [7, 6, 8, 2] and code[0, 32] == 5       # 3 + 2^-21 over 2^1
    code, s = mx_ref.quantize(x, mx_ref.MXFP8)
    assert list(s[0]) == [127 - 6, 127 - 6, 0] and mx_ref.values(code, s, 1)[0, 1] == 5.0
    x[0, 40] = np.inf
    assert list(mx_ref.quantize(x, mx_ref.MXFP4)[1][0]) == [127, 255, 0]
    p = mx_ref.pack(np.array([[2, 15]], np.uint8))
    assert p[0, 0] == 0xF2 and list(mx_ref.unpack(p)[0]) == [2, 15]
    # torch's e4m3 names the same values
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, mx_ref.E4M3)


def test_library_exports_the_header():
    declared = k3mx.declared_symbols(HEADER)
    assert declared == ["k3mx_mx_dequantize", "k3mx_mx_grouped", "k3mx_mx_linear", "k3mx_mx_quantize",
                        "k3mx_rmsnorm_mx"]
    out = subprocess.run(["nm", "-D", "--defined-only", k3mx.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert set(declared) <= set(re.findall(r"\sT\s(k3mx_\w+)", out))
    for name in declared:
        assert callable(getattr(k3mx, name))


def call(func, ok, order, **kw):
    return getattr(k3mx.lib(), func)(*(dict(ok, **kw)[k] for k in order.split()), None)


def test_quantize_refuses_bad_arguments():
    ok = dict(q=FAKE, s=FAKE, x=FAKE, dt=1, r=4, c=64, ld=64, f=0)
    go = lambda **kw: call("k3mx_mx_quantize", ok, "q s x dt r c ld f", **kw)
    assert go(q=None) == 1 and go(s=None) == 1 and go(x=None) == 1
    assert go(dt=2) == 1 and go(f=2) == 1 and go(f=-1) == 1
    assert go(r=0) == 3 and go(c=48) == 3 and go(c=0) == 3 and go(ld=63) == 3
    assert go(r=(1 << 24) + 1) == 3 and go(c=(1 << 20) + 32, ld=1 << 21) == 3
    assert go(r=1 << 24, c=1 << 20, ld=1 << 20) == 3           # too many elements
    assert go(q=FAKE + 8) == 2 and go(x=FAKE + 1) == 2 and go(dt=0, x=FAKE + 2) == 2


def test_dequantize_refuses_bad_arguments():
    ok = dict(y=FAKE, dt=1, q=FAKE, s=FAKE, r=4, c=64, f=0)
    go = lambda **kw: call("k3mx_mx_dequantize", ok, "y dt q s r c f", **kw)
    assert go(y=None) == 1 and go(q=None) == 1 and go(s=None) == 1 and go(dt=3) == 1 and go(f=2) == 1
    assert go(r=0) == 3 and go(c=33) == 3
    assert go(y=FAKE + 4) == 2 and go(q=FAKE + 4) == 2


def test_norm_refuses_bad_arguments():
    ok = dict(q=FAKE, s=FAKE, sum=FAKE, n=None, x=FAKE, ld=64, r=FAKE, dt=1, g=FAKE, eps=1e-5, t=2, w=64)
    go = lambda **kw: call("k3mx_rmsnorm_mx", ok, "q s sum n x ld r dt g eps t w", **kw)
    assert go(q=None) == 1 and go(g=None) == 1 and go(dt=2) == 1
    assert go(sum=None) == 1 and go(r=None) == 1                # both or neither
    assert go(eps=-1e-5) == 1 and go(eps=float("nan")) == 1 and go(eps=float("inf")) == 1
    assert go(t=0) == 3 and go(w=40) == 3 and go(ld=32) == 3 and go(w=32768 + 32, ld=65536) == 3
    assert go(x=FAKE + 2) == 2 and go(ld=68) == 2 and go(n=FAKE + 2) == 2 and go(g=FAKE + 4) == 2


@pytest.mark.parametrize("func", ["k3mx_mx_linear", "k3mx_mx_grouped"])
def test_products_refuse_bad_arguments(func):
    ok = dict(y=FAKE, dt=0, q=FAKE, s=FAKE, p=FAKE, ws=FAKE, off=FAKE, E=2, t=3, k=256, n=5)
    order = "y dt q s p ws t k n" if func == "k3mx_mx_linear" else "y dt q s p ws off E t k n"
    go = lambda **kw: call(func, ok, order, **kw)
    for k in ("y", "q", "s", "p", "ws"):
        assert go(**{k: None}) == 1
    assert go(dt=2) == 1
    assert go(t=0) == 3 and go(n=0) == 3 and go(k=64) == 3 and go(k=320) == 3 and go(k=65536 + 128) == 3
    assert go(y=FAKE + 4) == 2 and go(q=FAKE + 8) == 2 and go(p=FAKE + 16) == 2
    assert go(s=FAKE + 2) == 2 and go(ws=FAKE + 1) == 2
    if func == "k3mx_mx_grouped":
        assert go(off=None) == 1 and go(off=FAKE + 2) == 2
        assert go(E=0) == 3 and go(E=1025) == 3 and go(E=1024, n=1 << 21) == 3


def test_binding_refuses_mismatched_shapes():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    f32 = lambda *s: torch.zeros(*s, dtype=torch.float32)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    shape = [
        lambda: k3mx.k3mx_mx_quantize(u8(2, 32), u8(2, 2), f32(2, 96), k3mx.K3MX_MXFP4),
        lambda: k3mx.k3mx_mx_quantize(u8(2, 64), u8(2, 1), f32(2, 64), k3mx.K3MX_MXFP8),
        lambda: k3mx.k3mx_mx_quantize(u8(2, 48), u8(2, 1), f32(2, 48), k3mx.K3MX_MXFP8),
        lambda: k3mx.k3mx_mx_quantize(u8(64, 2), u8(64, 1), f32(2, 64).T, k3mx.K3MX_MXFP4),
        lambda: k3mx.k3mx_mx_quantize(u8(2, 64), u8(2, 2), f32(1, 64).expand(2, 64), k3mx.K3MX_MXFP8),
        lambda: k3mx.k3mx_mx_quantize(u8(0, 64), u8(0, 2), f32(0, 64), k3mx.K3MX_MXFP8),
        lambda: k3mx.k3mx_mx_dequantize(f32(2, 64), u8(2, 64), u8(2, 2), k3mx.K3MX_MXFP4),
        lambda: k3mx.k3mx_rmsnorm_mx(u8(2, 64), u8(2, 2), f32(2, 64), f32(2, 64), f32(1, 64), bf(64), 1e-5),
        lambda: k3mx.k3mx_rmsnorm_mx(u8(2, 64), u8(2, 2), None, f32(2, 64), f32(2, 64), bf(64), 1e-5),
        lambda: k3mx.k3mx_rmsnorm_mx(u8(2, 64), u8(2, 2), None, f32(2, 64), None, bf(32), 1e-5),
        lambda: k3mx.k3mx_mx_linear(f32(2, 5), u8(3, 128), u8(3, 4), u8(5, 64), u8(5, 4)),
        lambda: k3mx.k3mx_mx_linear(f32(3, 5), u8(3, 128), u8(3, 4), u8(6, 64), u8(6, 4)),
        lambda: k3mx.k3mx_mx_linear(f32(3, 5), u8(3, 128), u8(3, 4), u8(5, 64), u8(5, 2)),
        lambda: k3mx.k3mx_mx_grouped(f32(3, 5), u8(3, 128), u8(3, 4), u8(3, 5, 64), u8(2, 5, 4), off),
        lambda: k3mx.k3mx_mx_grouped(f32(3, 5), u8(3, 128), u8(3, 4), u8(2, 5, 64), u8(2, 5, 4), off[:1]),
    ]
    for i, go in enumerate(shape):
        with pytest.raises(TypeError) as err:
            go()
        assert "CUDA" not in str(err.value), (i, str(err.value))
    with pytest.raises(ValueError, match="fmt"):
        k3mx.k3mx_mx_quantize(u8(2, 64), u8(2, 2), f32(2, 64), 7)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        k3mx.k3mx_mx_quantize(u8(2, 64), u8(2, 2), f32(2, 64).half(), k3mx.K3MX_MXFP8)
    with pytest.raises(TypeError, match="CUDA"):
        k3mx.k3mx_mx_linear(f32(3, 5), u8(3, 128), u8(3, 4), u8(5, 64), u8(5, 4))
    with pytest.raises(TypeError, match="CUDA"):
        k3mx.k3mx_mx_grouped(f32(3, 5), u8(3, 128), u8(3, 4), u8(2, 5, 64), u8(2, 5, 4), off)


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU behaviour only")
def test_valid_call_without_gpu_fails_loudly():
    assert k3mx.lib().k3mx_mx_linear(FAKE, 0, FAKE, FAKE, FAKE, FAKE, 3, 256, 5, None) in (5, 7)
