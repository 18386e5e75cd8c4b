"""The steps of an expert block without a GPU: the definitions against
differences and by hand, exported symbols, and the refusals of the C ABI and of
the binding."""
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import block_ref
import mxfp4_routed_expert_k3mx_gb300 as k3mx

FAKE = 0x10000
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "k3mx_block.h")
FILES = ("block.cu", "situ.cu")


def test_sort_by_hand():
    offsets, perm, place = block_ref.sort(np.array([[2, 0], [-1, 2], [0, 2]]), 4)
    assert list(offsets) == [0, 2, 2, 5, 5] and list(perm) == [1, 4, 0, 3, 5]
    assert place.tolist() == [[2, 0], [-1, 3], [1, 4]]


def test_gradients_are_the_definitions_differences():
    r = np.random.default_rng(0)
    rows, place, w, dy = r.normal(size=(5, 7)), np.array([[0, 3], [-1, 4], [1, 2]]), r.normal(size=(3, 2)), r.normal(size=(3, 7))
    dr, dw, _ = block_ref.combine_backward(dy, rows, place, w)
    f = lambda rows, w: (block_ref.combine(rows, place, w, None)[0] * dy).sum()
    h = 1e-5
    for t, k in np.argwhere(place >= 0):
        e = np.zeros_like(w)
        e[t, k] = h
        assert abs((f(rows, w + e) - f(rows, w - e)) / (2 * h) - dw[t, k]) < 1e-8
        e = np.zeros_like(rows)
        e[place[t, k], 3] = h
        assert abs((f(rows + e, w) - f(rows - e, w)) / (2 * h) - dr[t, k, 3]) < 1e-8
    g, u, dh = r.normal(size=50) * 5, r.normal(size=50) * 20, r.normal(size=50)
    dg, du, _ = block_ref.situ_backward(g, u, dh)
    assert np.allclose((block_ref.situ(g + h, u) - block_ref.situ(g - h, u)) / (2 * h) * dh, dg, rtol=0, atol=1e-7)
    assert np.allclose((block_ref.situ(g, u + h) - block_ref.situ(g, u - h)) / (2 * h) * dh, du, rtol=0, atol=1e-7)
    x, dn, gain, dres = r.normal(size=(3, 8)), r.normal(size=(3, 8)), r.normal(size=8), r.normal(size=(3, 8))
    dx, dg, _, _ = block_ref.norm_backward(x, dn, gain, 0.1, dres)
    n = lambda x, gain: (x * gain / np.sqrt((x * x).mean(1, keepdims=True) + 0.1) * dn).sum() + (x * dres).sum()
    for i in range(3):
        for j in range(8):
            e = np.zeros_like(x)
            e[i, j] = h
            assert abs((n(x + e, gain) - n(x - e, gain)) / (2 * h) - dx[i, j]) < 1e-8
            assert abs((n(x, gain + e[i]) - n(x, gain - e[i])) / (2 * h) - dg[j]) < 1e-8


def test_library_exports_the_header():
    declared = k3mx.declared_symbols(HEADER)
    assert declared == sorted([*k3mx._BLOCK_FUNCS, "k3mx_sort_workspace_size", "k3mx_rmsnorm_mx_backward_workspace_size"])
    out = subprocess.run(["nm", "-D", "--defined-only", k3mx.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert set(declared) <= set(re.findall(r"\sT\s(k3mx_\w+)", out))
    for name in declared:
        assert callable(getattr(k3mx, name))


@pytest.mark.parametrize("name", FILES)
def test_kernels_wait_and_read_as_they_should(name):
    """Inputs may be what the kernel ahead writes: every kernel waits for it
    before its first load, and none reads through the read-only path."""
    text = open(os.path.join(os.path.dirname(k3mx.LIB_PATH), "csrc", name)).read()
    text = re.sub(r"/\*.*?\*/", "", re.sub(r"//[^\n]*", "", text), flags=re.S)
    for word in ("__ldg", "ld.global.nc", "__restrict__"):
        assert word not in text, word
    kernels = text.split("__global__")[1:]
    assert len(kernels) >= 4
    for k in kernels:
        assert "pdl_wait()" in k and k.index("pdl_wait()") < k.index("pdl_launch_dependents()")


def call(func, ok, order, **kw):
    return getattr(k3mx.lib(), func)(*(dict(ok, **kw)[k] for k in order.split()), None)


def test_workspace_sizes():
    assert k3mx.k3mx_sort_workspace_size(0, 1, 1) == 0 and k3mx.k3mx_sort_workspace_size(1, 1, 1025) == 0
    assert k3mx.k3mx_sort_workspace_size(1, 16, 896) == 0                   # few pairs need none
    big = k3mx.k3mx_sort_workspace_size(65536, 16, 896)
    assert 0 < big < 64 << 20 and big % 256 == 0
    size = k3mx.k3mx_rmsnorm_mx_backward_workspace_size
    assert size(0, 64) == 0 and size(4, 48) == 0 and size(4, 32768 + 32) == 0
    assert size(1, 64) > 0 and size(8192, 16384) <= 64 << 20
    assert size(1 << 24, 64) >= (1 << 24) // 8 // 1024 * 64 * 4             # no thread adds more than 1024 rows


def test_sort_refuses_bad_arguments():
    ok = dict(o=FAKE, p=FAKE, l=FAKE, i=FAKE, t=4096, k=16, e=896, ws=FAKE, n=1 << 24)
    go = lambda **kw: call("k3mx_sort", ok, "o p l i t k e ws n", **kw)
    assert go(o=None) == 1 and go(l=None) == 1 and go(i=None) == 1
    for kw in (dict(t=0), dict(k=0), dict(t=-1), dict(t=1 << 20, k=17), dict(e=0), dict(e=1025), dict(t=1 << 30, k=1 << 30)):
        assert go(**kw) == 3, kw
    for key in "opli":
        assert go(**{key: FAKE + 2}) == 2
    assert go(ws=None) == 4 and go(n=k3mx.k3mx_sort_workspace_size(4096, 16, 896) - 1) == 4 and go(ws=FAKE + 8) == 2


def test_dispatch_refuses_bad_arguments():
    ok = dict(r=FAKE, s=None, x=FAKE, xs=None, ld=64, dt=1, p=FAKE, t=4, k=2, n=8, w=64)
    go = lambda **kw: call("k3mx_dispatch", ok, "r s x xs ld dt p t k n w", **kw)
    assert go(r=None) == 1 and go(x=None) == 1 and go(p=None) == 1 and go(dt=3) == 1 and go(dt=-1) == 1
    assert go(s=FAKE) == 1 and go(xs=FAKE) == 1 and go(s=FAKE, xs=FAKE) == 1 and go(dt=2) == 1 and go(dt=2, s=FAKE) == 1
    assert go(t=0) == 3 and go(k=0) == 3 and go(n=0) == 3 and go(w=0) == 3 and go(ld=63) == 3 and go(ld=(1 << 32) + 1) == 3
    assert go(t=1 << 24, k=2) == 3 and go(n=(1 << 24) + 1) == 3 and go(w=(1 << 20) + 1, ld=1 << 21) == 3
    assert go(n=1 << 19, w=1 << 20, ld=1 << 20) == 3 and go(t=1 << 19, w=1 << 20, ld=1 << 20) == 3
    assert go(dt=2, s=FAKE, xs=FAKE, w=48, ld=48) == 3
    assert go(r=FAKE + 1) == 2 and go(x=FAKE + 1) == 2 and go(dt=0, x=FAKE + 2) == 2 and go(p=FAKE + 2) == 2


def test_combine_refuses_bad_arguments():
    ok = dict(y=FAKE, yt=0, r=FAKE, rt=1, p=FAKE, w=FAKE, b=FAKE, t=4, k=2, n=8, c=64)
    go = lambda **kw: call("k3mx_combine", ok, "y yt r rt p w b t k n c", **kw)
    assert go(y=None) == 1 and go(r=None) == 1 and go(p=None) == 1 and go(yt=2) == 1 and go(rt=2) == 1
    assert go(t=0) == 3 and go(k=0) == 3 and go(n=0) == 3 and go(c=0) == 3 and go(n=1 << 19, c=1 << 20) == 3
    assert go(y=FAKE + 2) == 2 and go(b=FAKE + 2) == 2 and go(r=FAKE + 1) == 2 and go(p=FAKE + 1) == 2 and go(w=FAKE + 2) == 2
    ok = dict(dr=FAKE, dw=FAKE, dy=FAKE, ld=64, dt=1, r=FAKE, rt=0, p=FAKE, w=FAKE, t=4, k=2, n=8, c=64)
    go = lambda **kw: call("k3mx_combine_backward", ok, "dr dw dy ld dt r rt p w t k n c", **kw)
    for key in ("dr", "dw", "dy", "r", "p", "w"):
        assert go(**{key: None}) == 1
    assert go(dt=2) == 1 and go(rt=2) == 1
    assert go(t=0) == 3 and go(k=0) == 3 and go(n=0) == 3 and go(c=0) == 3 and go(ld=63) == 3 and go(ld=(1 << 32) + 1) == 3
    assert go(dr=FAKE + 2) == 2 and go(dw=FAKE + 2) == 2 and go(dy=FAKE + 1) == 2 and go(r=FAKE + 2) == 2


def test_activation_refuses_bad_arguments():
    ok = dict(q=FAKE, s=FAKE, v=FAKE, vs=FAKE, x=FAKE, ld=128, dt=1, r=4, f=64)
    go = lambda **kw: call("k3mx_situ_mx", ok, "q s v vs x ld dt r f", **kw)
    assert go(q=None) == 1 and go(s=None) == 1 and go(x=None) == 1 and go(v=None) == 1 and go(vs=None) == 1 and go(dt=2) == 1
    assert go(r=0) == 3 and go(f=48) == 3 and go(f=0) == 3 and go(ld=120) == 3 and go(f=(1 << 19) + 32, ld=1 << 21) == 3
    assert go(q=FAKE + 8) == 2 and go(v=FAKE + 8) == 2 and go(x=FAKE + 8) == 2 and go(ld=132) == 2
    ok = dict(d=FAKE, h=FAKE, ld=64, dt=1, v=FAKE, vs=FAKE, r=4, f=64)
    go = lambda **kw: call("k3mx_situ_mx_backward", ok, "d h ld dt v vs r f", **kw)
    for key in ("d", "h", "v", "vs"):
        assert go(**{key: None}) == 1
    assert go(dt=2) == 1 and go(r=0) == 3 and go(f=40) == 3 and go(ld=63) == 3
    assert go(d=FAKE + 8) == 2 and go(h=FAKE + 4) == 2 and go(v=FAKE + 8) == 2 and go(ld=68) == 2


def test_norm_backward_refuses_bad_arguments():
    need = k3mx.k3mx_rmsnorm_mx_backward_workspace_size(4, 64)
    ok = dict(dx=FAKE, dw=FAKE, dn=FAKE, ld=64, dr=FAKE, dt=1, v=FAKE, vs=FAKE, g=FAKE, eps=1e-5, t=4, w=64, ws=FAKE, n=need)
    go = lambda **kw: call("k3mx_rmsnorm_mx_backward", ok, "dx dw dn ld dr dt v vs g eps t w ws n", **kw)
    for key in ("dx", "dw", "dn", "v", "vs", "g"):
        assert go(**{key: None}) == 1
    assert go(dt=2) == 1 and go(eps=-1.0) == 1 and go(eps=float("nan")) == 1 and go(eps=float("inf")) == 1
    assert go(t=0) == 3 and go(w=40) == 3 and go(ld=63) == 3 and go(w=32768 + 32, ld=65536) == 3
    for key in ("dx", "dw", "dn", "dr", "v", "g", "ws"):
        assert go(**{key: FAKE + 8}) == 2
    assert go(ld=68) == 2 and go(ws=None) == 4 and go(n=need - 1) == 4


def test_binding_names_what_is_wrong():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    f32 = lambda *s: torch.zeros(*s)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    bad = [
        ("idx", lambda: k3mx.k3mx_sort(i32(5), i32(6), i32(3, 2), i32(6), None)),
        ("offsets", lambda: k3mx.k3mx_sort(i32(1), i32(6), i32(3, 2), i32(3, 2), None)),
        ("place", lambda: k3mx.k3mx_sort(i32(5), i32(6), i32(2, 3), i32(3, 2), None)),
        ("perm", lambda: k3mx.k3mx_sort(i32(5), i32(5), i32(3, 2), i32(3, 2), None)),
        ("x", lambda: k3mx.k3mx_dispatch(f32(6, 8), f32(3, 8).double(), i32(3, 2))),
        ("rows", lambda: k3mx.k3mx_dispatch(f32(6, 9), f32(3, 8), i32(3, 2))),
        ("place", lambda: k3mx.k3mx_dispatch(f32(6, 8), f32(3, 8), i32(2, 3))),
        ("x", lambda: k3mx.k3mx_dispatch(u8(6, 48), u8(3, 48), i32(3, 2), u8(6, 1), u8(3, 1))),
        ("scales", lambda: k3mx.k3mx_dispatch(u8(6, 64), u8(3, 64), i32(3, 2))),
        ("scales, x_scales", lambda: k3mx.k3mx_dispatch(f32(6, 64), f32(3, 64), i32(3, 2), u8(6, 2), u8(3, 2))),
        ("x", lambda: k3mx.k3mx_dispatch(f32(6, 8), f32(1, 8).expand(3, 8), i32(3, 2))),
        ("rows", lambda: k3mx.k3mx_combine(f32(3, 8), f32(6, 7), i32(3, 2))),
        ("w", lambda: k3mx.k3mx_combine(f32(3, 8), f32(6, 8), i32(3, 2), w=f32(2, 3))),
        ("base", lambda: k3mx.k3mx_combine(f32(3, 8), f32(6, 8), i32(3, 2), base=f32(3, 9))),
        ("y", lambda: k3mx.k3mx_combine(f32(3, 16)[:, ::2], f32(6, 8), i32(3, 2))),
        ("y", lambda: k3mx.k3mx_combine(f32(3, 9)[:, :8], f32(6, 8), i32(3, 2))),
        ("y", lambda: k3mx.k3mx_combine(f32(0, 8), f32(6, 8), i32(0, 2))),
        ("drows", lambda: k3mx.k3mx_combine_backward(f32(5, 8), f32(3, 2), f32(3, 8), f32(6, 8), i32(3, 2), f32(3, 2))),
        ("dw", lambda: k3mx.k3mx_combine_backward(f32(6, 8), f32(2, 3), f32(3, 8), f32(6, 8), i32(3, 2), f32(3, 2))),
        ("gu", lambda: k3mx.k3mx_situ_mx(u8(2, 48), u8(2, 1), f32(2, 96))),
        ("codes", lambda: k3mx.k3mx_situ_mx(u8(2, 64), u8(2, 1), f32(2, 64))),
        ("saved_scales", lambda: k3mx.k3mx_situ_mx(u8(2, 32), u8(2, 1), f32(2, 64), saved=u8(2, 64))),
        ("saved", lambda: k3mx.k3mx_situ_mx(u8(2, 32), u8(2, 1), f32(2, 64), saved=u8(2, 32), saved_scales=u8(2, 2))),
        ("dgu", lambda: k3mx.k3mx_situ_mx_backward(f32(2, 32), f32(2, 32), u8(2, 64), u8(2, 2))),
        ("saved", lambda: k3mx.k3mx_situ_mx_backward(f32(2, 64), f32(2, 32), u8(2, 32), u8(2, 2))),
        ("dweight", lambda: k3mx.k3mx_rmsnorm_mx_backward(f32(2, 32), f32(31), f32(2, 32), u8(2, 32), u8(2, 1), bf(32), 1e-5, None)),
        ("dres", lambda: k3mx.k3mx_rmsnorm_mx_backward(f32(2, 32), f32(32), f32(2, 32), u8(2, 32), u8(2, 1), bf(32), 1e-5, None,
                                                       dres=f32(2, 31))),
        ("dn", lambda: k3mx.k3mx_rmsnorm_mx_backward(f32(2, 40), f32(40), f32(2, 40), u8(2, 40), u8(2, 1), bf(40), 1e-5, None)),
    ]
    for i, (name, go) in enumerate(bad):
        with pytest.raises(TypeError) as err:
            go()
        assert str(err.value).startswith(name + ":") and "CUDA" not in str(err.value), (i, str(err.value))
    with pytest.raises(TypeError, match="CUDA"):
        k3mx.k3mx_combine(f32(3, 8), f32(6, 8), i32(3, 2))
    with pytest.raises(TypeError, match="CUDA"):
        k3mx.k3mx_situ_mx_backward(f32(2, 64), f32(2, 32), u8(2, 64), u8(2, 2))


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU behaviour only")
def test_valid_call_without_gpu_fails_loudly():
    assert k3mx.lib().k3mx_combine(FAKE, 0, FAKE, 0, FAKE, None, None, 3, 2, 6, 64, None) in (5, 7)
