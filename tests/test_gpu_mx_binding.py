"""The microscaled operators' Python calls with device tensors: what is
accepted, what is refused, and first calls from several threads."""
import os
import subprocess
import sys

import pytest
import torch

import mxfp4_routed_expert_k3mx_gb300 as k3mx

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def tensors():
    u8 = lambda *s: torch.randint(0, 100, s, dtype=torch.uint8, device="cuda:0")
    f = lambda *s, dtype=torch.bfloat16: torch.randn(*s, device="cuda:0").to(dtype)
    return {
        "k3mx_mx_quantize": dict(codes=u8(4, 128), scales=u8(4, 4), x=f(4, 128), fmt=k3mx.K3MX_MXFP8),
        "k3mx_mx_dequantize": dict(y=f(4, 128), codes=u8(4, 64), scales=u8(4, 4), fmt=k3mx.K3MX_MXFP4),
        "k3mx_rmsnorm_mx": dict(codes=u8(4, 128), scales=u8(4, 4), sum=f(4, 128), x=f(4, 128), residual=f(4, 128),
                                weight=f(128), eps=1e-5, normed=f(4, 128)),
        "k3mx_mx_linear": dict(y=f(4, 128), codes=u8(4, 256), scales=u8(4, 8), packed=u8(128, 128), wscales=u8(128, 8)),
        "k3mx_mx_grouped": dict(y=f(4, 128), codes=u8(4, 256), scales=u8(4, 8), packed=u8(2, 128, 128), wscales=u8(2, 128, 8),
                                offsets=torch.tensor([0, 1, 4], dtype=torch.int32, device="cuda:0")),
    }


@pytest.mark.parametrize("name", sorted(k3mx._MX_FUNCS))
def test_each_argument_is_checked(cuda_dev, name):
    """A call with one argument on the host, of another type, one element
    longer, of other strides or no tensor at all is refused before anything is launched."""
    ok = tensors()[name]
    call = getattr(k3mx, name)
    call(**ok)
    for key, t in ok.items():
        if not isinstance(t, torch.Tensor):
            continue
        bad = [t.cpu(), t.to(torch.float16), torch.cat([t, t[:1]]), t.unsqueeze(0), 3, t.to_sparse()]
        if key != "x" and t.dim() > 1:
            bad.append(torch.cat([t, t], -1)[..., :t.shape[-1]])             # row pitch
        if t.dim() > 1:
            bad += [torch.empty_like(t.transpose(-1, -2).contiguous()).transpose(-1, -2), t[:0]]
        if key not in ("sum", "residual", "normed"):
            bad.append(None)
        for v in bad:
            with pytest.raises((TypeError, ValueError, AttributeError)):
                call(**dict(ok, **{key: v}))
    for key, v in (("fmt", 2), ("fmt", -1), ("fmt", "mxfp8"), ("eps", "small"), ("eps", None)):
        if key in ok:
            with pytest.raises((TypeError, ValueError)):
                call(**dict(ok, **{key: v}))
    torch.cuda.synchronize()
    assert k3mx.k3mx_device_status() == (0, 0)
    call(**ok)


def test_forms_of_tensors_that_are_taken(cuda_dev):
    """Rows apart, one row of any pitch, parameters, tensors that need a
    gradient; refusals of the library itself keep their names."""
    a = tensors()["k3mx_mx_quantize"]
    want = [t.clone() for t in k3mx.k3mx_mx_quantize(**a)]
    wide = torch.zeros(4, 160, dtype=torch.bfloat16, device="cuda:0")
    wide[:, :128] = a["x"]
    for x in (wide[:, :128], torch.nn.Parameter(a["x"].clone()), a["x"].clone().requires_grad_()):
        got = k3mx.k3mx_mx_quantize(a["codes"].fill_(0), a["scales"].fill_(0), x, True)       # an int by another name
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    one = torch.zeros(1, 128, dtype=torch.bfloat16, device="cuda:0").as_strided((1, 128), (1, 1))
    one.copy_(a["x"][:1])
    got = k3mx.k3mx_mx_quantize(a["codes"][:1], a["scales"][:1], one, k3mx.K3MX_MXFP8)
    assert torch.equal(got[0], want[0][:1])
    b = tensors()["k3mx_mx_linear"]
    off = torch.empty(4 * 256 + 1, dtype=torch.uint8, device="cuda:0")[1:].view(4, 256)
    with pytest.raises(k3mx.K3mxError, match="K3MX_EALIGN"):
        k3mx.k3mx_mx_linear(**dict(b, codes=off))


def test_first_calls_from_several_threads(cuda_dev):
    """Four threads of a fresh process make the first calls at once, each on its
    own stream."""
    code = """
import threading, torch
import mxfp4_routed_expert_k3mx_gb300 as k3mx
x = torch.randn(64, 7168, device="cuda:0").to(torch.bfloat16)
go, out = threading.Barrier(4), [None] * 4
def work(i):
    with torch.cuda.stream(torch.cuda.Stream()):
        c = torch.empty(64, 7168, dtype=torch.uint8, device="cuda:0"); s = torch.empty(64, 224, dtype=torch.uint8, device="cuda:0")
        w = torch.empty(128, 3584, dtype=torch.uint8, device="cuda:0"); ws = torch.empty(128, 224, dtype=torch.uint8, device="cuda:0")
        y = torch.empty(64, 128, device="cuda:0")
        torch.cuda.synchronize()
        go.wait()
        for _ in range(50):
            k3mx.k3mx_mx_quantize(c, s, x, k3mx.K3MX_MXFP8)
            k3mx.k3mx_mx_quantize(w, ws, torch.cat([x, x]), k3mx.K3MX_MXFP4)
            k3mx.k3mx_mx_linear(y, c, s, w, ws)
        torch.cuda.current_stream().synchronize()
        out[i] = y
ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
[t.start() for t in ts]; [t.join() for t in ts]
assert all(o is not None and torch.equal(o, out[0]) for o in out)
assert k3mx.k3mx_device_status() == (0, 0)
print("same")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=240)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr
