"""The steps of an expert block together, forward and backward, as a program
runs them: stage by stage, captured, on other streams, from two threads; and
what the Python calls take and refuse of device tensors."""
import importlib.util
import os
import threading

import numpy as np
import pytest
import torch

import block_ref
import mx_ref
import mxfp4_routed_expert_k3mx_gb300 as k3mx
from test_gpu_mx_device import Elsewhere

pytestmark = pytest.mark.gpu
DEV = "cuda"
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block_train.py")


@pytest.fixture(scope="module")
def example(cuda_dev):
    spec = importlib.util.spec_from_file_location("moe_block_train", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def doubles(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("tokens,topk,experts", [(1, 1, 1), (1, 4, 16), (65, 3, 16), (300, 4, 40)])
def test_a_step_of_the_example(example, tokens, topk, experts):
    """Every stage against its definition applied to what the one before wrote."""
    block = example.Block(hidden=256, experts=experts, topk=topk, inter=128, seed=tokens)
    gen = torch.Generator(device=DEV).manual_seed(tokens)
    x, res, dy = (torch.randn(tokens, 256, generator=gen, device=DEV) for _ in range(3))
    b = block.buffers(tokens)
    y = block.forward(x, res, b)
    block.backward(dy, b)
    assert k3mx.k3mx_device_status() == (0, 0)
    r = {k: v.cpu().numpy() if v.dtype in (torch.uint8, torch.int32) else doubles(v) for k, v in b.items()}
    F = 128
    offsets, perm, place = block_ref.sort(r["idx"], experts)
    assert np.array_equal(r["offsets"], offsets) and np.array_equal(r["perm"], perm) and np.array_equal(r["place"], place)
    token = perm // topk
    assert np.array_equal(r["rows"], r["codes"][token]) and np.array_equal(r["row_scales"], r["scales"][token])
    for codes, scales, of in (("kept", "kept_scales", "sum"), ("saved", "saved_scales", "gu")):
        c, s = mx_ref.quantize(r[of], mx_ref.MXFP8)
        assert np.array_equal(c, r[codes]) and np.array_equal(s, r[scales])
    c, s = mx_ref.quantize(block_ref.situ(r["gu"][:, :F], r["gu"][:, F:]), mx_ref.MXFP8)
    assert np.array_equal(s, r["h_scales"]) and np.array_equal(c, r["h"])
    want, mag = block_ref.combine(r["out"], place, r["w"], r["sum"])
    assert np.all(np.abs(doubles(y) - want) <= (2 * topk + 3) * 2.0 ** -24 * mag)
    dr, dw, mag = block_ref.combine_backward(doubles(dy), r["out"], place, r["w"])
    assert np.all(np.abs(r["dout"][place] - dr) <= 2.0 ** -23 * np.abs(dr))
    assert np.all(np.abs(r["dw"] - dw) <= 24 * 2.0 ** -24 * mag)
    v = mx_ref.values(r["saved"], r["saved_scales"], mx_ref.MXFP8)
    dg, du, mag = block_ref.situ_backward(v[:, :F], v[:, F:], r["dh"])
    off = 2.0 ** -18 * (1 + (np.abs(v[:, :F]) + np.abs(v[:, F:])) / 16) + 2.0 ** -23
    assert np.all(np.abs(r["dgu"][:, :F] - dg) <= off * mag + 1e-30) and np.all(np.abs(r["dgu"][:, F:] - du) <= off * np.abs(du) + 1e-30)
    want, mag = block_ref.combine(r["drows"], place, None, None)
    rest = r["dlogits"] @ doubles(block.router)
    tol = (2 * topk + 3) * 2.0 ** -24 * mag + (experts + 4) * 2.0 ** -23 * (np.abs(r["dlogits"]) @ np.abs(doubles(block.router)) + mag)
    assert np.all(np.abs(r["dn"] - want - rest) <= tol)
    wx, wg, mx, mg = block_ref.norm_backward(mx_ref.values(r["kept"], r["kept_scales"], mx_ref.MXFP8), r["dn"], doubles(block.gain),
                                             np.float64(np.float32(example.EPS)), doubles(dy))
    assert np.all(np.abs(r["dx"] - wx) <= 64 * 2.0 ** -24 * mx) and np.all(np.abs(r["dgain"] - wg) <= 200 * 2.0 ** -24 * mg)


def own_calls(block, b, x, res, dy):
    """The library's calls of a step (the choices are given)."""
    k3mx.k3mx_rmsnorm_mx(b["codes"], b["scales"], b["sum"], x, res, block.gain, 1e-5, normed=b["normed"])
    k3mx.k3mx_mx_quantize(b["kept"], b["kept_scales"], b["sum"], k3mx.K3MX_MXFP8)
    k3mx.k3mx_sort(b["offsets"], b["perm"], b["place"], b["idx"], b["workspace"])
    k3mx.k3mx_dispatch(b["rows"], b["codes"], b["place"], scales=b["row_scales"], x_scales=b["scales"])
    k3mx.k3mx_mx_grouped(b["gu"], b["rows"], b["row_scales"], *block.w13[:2], b["offsets"])
    k3mx.k3mx_situ_mx(b["h"], b["h_scales"], b["gu"], saved=b["saved"], saved_scales=b["saved_scales"])
    k3mx.k3mx_mx_grouped(b["out"], b["h"], b["h_scales"], *block.w2[:2], b["offsets"])
    k3mx.k3mx_combine(b["y"], b["out"], b["place"], w=b["w"], base=b["sum"])
    k3mx.k3mx_combine_backward(b["dout"], b["dw"], dy, b["out"], b["place"], b["w"])
    k3mx.k3mx_situ_mx_backward(b["dgu"], b["dout"][:, :block.inter], b["saved"], b["saved_scales"])
    k3mx.k3mx_combine(b["dn"], b["out"], b["place"])
    k3mx.k3mx_rmsnorm_mx_backward(b["dx"], b["dgain"], b["dn"], b["kept"], b["kept_scales"], block.gain, 1e-5, b["workspace"], dres=dy)


RESULTS = ("offsets", "perm", "place", "rows", "row_scales", "h", "h_scales", "saved", "saved_scales", "y", "dout", "dw", "dgu", "dn",
           "dx", "dgain")


def a_run(example, tokens, seed, block=None):
    block = block or example.Block(hidden=512, experts=16, topk=4, inter=128, seed=1)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    ins = [torch.randn(tokens, 512, generator=gen, device=DEV) for _ in range(3)]
    b = block.buffers(tokens)
    b["idx"] = torch.randint(-1, 16, (tokens, 4), generator=gen, device=DEV, dtype=torch.int32)
    b["w"] = torch.rand(tokens, 4, generator=gen, device=DEV)
    for k in ("perm", "rows", "row_scales", "dout", "out", "gu"):
        b[k].zero_()                                  # (rows behind the last are left as they are)
    return block, b, ins


@pytest.mark.parametrize("tokens", [1, 70, 1500])
def test_captured_and_replayed(example, tokens):
    block, b, ins = a_run(example, tokens, 1)
    own_calls(block, b, *ins)
    want = {k: b[k].clone() for k in RESULTS}
    own_calls(block, b, *ins)
    assert all(torch.equal(b[k], want[k]) for k in RESULTS)            # the same bits again
    # two graphs of other inputs that share the workspace, replayed in turn
    _, b2, ins2 = a_run(example, tokens, 2, block)
    b2["workspace"] = b["workspace"]
    own_calls(block, b2, *ins2)
    want2 = {k: b2[k].clone() for k in RESULTS}
    graphs = []
    for bb, ii in ((b, ins), (b2, ins2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            own_calls(block, bb, *ii)
        graphs.append(g)
    for k in RESULTS:
        for bb in (b, b2):
            if k not in ("perm", "rows", "row_scales", "dout"):
                bb[k].fill_(3)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(b[k], want[k]) and torch.equal(b2[k], want2[k]) for k in RESULTS)
    # new inputs in the same buffers
    for t, u in zip(ins, ins2):
        t.copy_(u)
    b["idx"].copy_(b2["idx"]), b["w"].copy_(b2["w"])
    graphs[0].replay()
    torch.cuda.synchronize()
    n = int(want2["offsets"][-1])
    for k in RESULTS:
        rows = slice(n if k in ("rows", "row_scales", "h", "h_scales", "saved", "saved_scales", "dout", "dgu") else None)
        a, c = (b[k][:n], want2[k][:n]) if k == "perm" else (b[k][rows], want2[k][rows])
        assert torch.equal(a, c), k
    assert k3mx.k3mx_device_status() == (0, 0)


def test_other_streams_and_threads(example):
    """Two threads, each on a stream of its own with its own buffers, and calls
    that name a stream."""
    block, b, ins = a_run(example, 700, 5)
    own_calls(block, b, *ins)
    want = {k: b[k].clone() for k in RESULTS}
    torch.cuda.synchronize()
    failed = []

    def work(seed):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                _, mine, mins = a_run(example, 700, 5, block)
                for _ in range(20):
                    own_calls(block, mine, *mins)
                s.synchronize()
                assert all(torch.equal(mine[k], want[k]) for k in RESULTS)
        except BaseException as e:          # noqa: B902 (a thread's own)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not failed, failed
    s = torch.cuda.Stream()
    y = torch.zeros_like(b["y"])
    s.wait_stream(torch.cuda.current_stream())
    k3mx.k3mx_combine(y, b["out"], b["place"], w=b["w"], base=b["sum"], stream=s)
    k3mx.k3mx_combine(y, b["out"], b["place"], w=b["w"], base=b["sum"], stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(y, want["y"])


def tensors():
    u8 = lambda *s: torch.randint(0, 100, s, dtype=torch.uint8, device="cuda:0")
    f = lambda *s, dtype=torch.bfloat16: torch.randn(*s, device="cuda:0").to(dtype)
    f32 = lambda *s: torch.randn(*s, device="cuda:0")
    place = torch.tensor([[0, 3], [1, 2], [-1, 4]], dtype=torch.int32, device="cuda:0")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda:0")
    return {
        "k3mx_sort": dict(offsets=i32(6), perm=i32(6), place=i32(3, 2), idx=place.clone(), workspace=u8(1 << 16)),
        "k3mx_dispatch": dict(rows=u8(5, 64), x=u8(3, 64), place=place, scales=u8(5, 2), x_scales=u8(3, 2)),
        "k3mx_combine": dict(y=f(3, 64), rows=f32(5, 64), place=place, w=f32(3, 2), base=f(3, 64)),
        "k3mx_combine_backward": dict(drows=f32(5, 64), dw=f32(3, 2), dy=f(3, 64), rows=f32(5, 64), place=place, w=f32(3, 2)),
        "k3mx_situ_mx": dict(codes=u8(3, 64), scales=u8(3, 2), gu=f(3, 128), saved=u8(3, 128), saved_scales=u8(3, 4)),
        "k3mx_situ_mx_backward": dict(dgu=f(3, 128), dh=f(3, 64), saved=u8(3, 128), saved_scales=u8(3, 4)),
        "k3mx_rmsnorm_mx_backward": dict(dx=f(3, 64), dweight=f32(64), dn=f(3, 64), saved=u8(3, 64), saved_scales=u8(3, 2), weight=f(64),
                                         eps=1e-5, workspace=u8(1 << 16), dres=f(3, 64)),
    }


OPTIONAL = {"perm", "workspace", "w", "base", "dres"}
STRIDED = {"x", "dy", "gu", "dh", "dn"}


@pytest.mark.parametrize("name", sorted(k3mx._BLOCK_FUNCS))
def test_each_argument_is_checked(cuda_dev, name):
    ok, call = tensors()[name], getattr(k3mx, name)
    call(**ok)
    for key, t in ok.items():
        if not isinstance(t, torch.Tensor):
            continue
        bad = [t.cpu(), 3, t.to_sparse()]
        if key != "workspace":
            bad += [t.to(torch.float16), torch.cat([t, t[:1]]) if key != "offsets" else t[:1]]
            if key != "perm":
                bad.append(t.unsqueeze(0))
        if key not in STRIDED and t.dim() > 1:
            bad.append(torch.cat([t, t], -1)[..., :t.shape[-1]])             # row pitch
        if t.dim() > 1:
            bad += [torch.empty_like(t.transpose(-1, -2).contiguous()).transpose(-1, -2), t[:0]]
        if key not in OPTIONAL or (key == "w" and name == "k3mx_combine_backward"):
            bad.append(None)
        for v in bad:
            if name in ("k3mx_dispatch", "k3mx_combine") and key == "rows" and isinstance(v, torch.Tensor) and v.shape[0] == 6:
                continue                                                      # (there may be as many rows as one likes)
            with pytest.raises((TypeError, ValueError, AttributeError)):
                call(**dict(ok, **{key: v}))
    for v in ("small", None):
        if "eps" in ok:
            with pytest.raises((TypeError, ValueError)):
                call(**dict(ok, eps=v))
    if "eps" in ok:
        with pytest.raises(k3mx.K3mxError, match="EINVAL"):
            call(**dict(ok, eps=-1.0))
        with pytest.raises(k3mx.K3mxError, match="EWORKSPACE"):
            call(**dict(ok, workspace=None))
    torch.cuda.synchronize()
    k3mx.k3mx_device_status()
    call(**ok)


@pytest.mark.parametrize("name", sorted(k3mx._BLOCK_FUNCS))
def test_a_tensor_of_another_device_is_named(cuda_dev, name):
    ok, call = tensors()[name], getattr(k3mx, name)
    for key, t in ok.items():
        if isinstance(t, torch.Tensor):
            with pytest.raises(TypeError, match=rf"^{key}: .*cuda:0.*cuda:1"):
                call(**dict(ok, **{key: Elsewhere(t)}))
    with pytest.raises(TypeError, match="cuda:1"):
        call(**{k: Elsewhere(t) if isinstance(t, torch.Tensor) else t for k, t in ok.items()})
    torch.cuda.synchronize()
    assert k3mx.k3mx_device_status() == (0, 0)


def test_forms_of_tensors_that_are_taken(cuda_dev):
    """One row of any pitch, tensors that need a gradient, inference tensors."""
    ok = tensors()["k3mx_combine_backward"]
    for dy in (torch.randn(3, 64, device=DEV).bfloat16().requires_grad_(), torch.randn(3, 71, device=DEV).bfloat16()[:, 5:69]):
        k3mx.k3mx_combine_backward(**dict(ok, dy=dy))
        want = (dy.detach().float() * ok["w"][:, 1:])[0]
        assert torch.allclose(ok["drows"][3], want)
    one = torch.randn(1, 200, device=DEV)[:, 8:72]
    with torch.inference_mode():
        rows = torch.zeros(2, 64, device=DEV)
        k3mx.k3mx_dispatch(rows, one, torch.tensor([[1]], dtype=torch.int32, device=DEV))
    assert torch.equal(rows[1], one[0]) and torch.all(rows[0] == 0)
