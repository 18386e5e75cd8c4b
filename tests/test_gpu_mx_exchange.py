"""Waits that give up in a cluster that still has exchanges ahead: several items
to a cluster, one or two exchanges each, so that both exchange barriers are used
again after the failure.  The call ends, says so, leaves nothing behind that
the launches right after it could meet, and the next calls are right."""
import pytest
import torch

import mxfp4_routed_expert_k3mx_gb300 as k3mx

pytestmark = pytest.mark.gpu


def product(rows, inner, out, dtype, groups=None):
    gen = torch.Generator(device="cuda:0").manual_seed(rows + out)
    u8 = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=gen, dtype=torch.uint8, device="cuda:0")
    x = (u8(0, 120, rows, inner), u8(120, 128, rows, inner // 32))
    lead = () if groups is None else (groups,)
    w = (u8(0, 255, *lead, out, inner // 2), u8(120, 128, *lead, out, inner // 32))
    y = torch.empty(rows, out, dtype=dtype, device="cuda:0")
    if groups is None:
        return y, lambda: k3mx.k3mx_mx_linear(y, *x, *w)
    off = torch.linspace(0, rows, groups + 1, device="cuda:0").round().to(torch.int32)
    return y, lambda: k3mx.k3mx_mx_grouped(y, *x, *w, off)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,inner,out,groups", [(2, 16384, 12800, None), (40, 65536, 5120, None), (64, 65536, 5120, None),
                                                   (64, 65536, 1280, 4)])
def test_exchanges_after_a_wait_gave_up(cuda_dev, dtype, rows, inner, out, groups):
    y, call = product(rows, inner, out, dtype, groups)
    call()
    assert k3mx.k3mx_device_status() == (0, 0)
    clean = y.clone()
    assert torch.isfinite(clean).all()
    k3mx.k3mx_set_wait_limit(1)
    try:
        seen = set()
        for i in range(12):
            for _ in range(1 + i % 3):
                call()
            seen.add(k3mx.k3mx_device_status())
    finally:
        k3mx.k3mx_set_wait_limit(0)
    assert all(st == 0 or st == 6 and 400 <= detail < 460 for st, detail in seen), seen
    # a poll lasts up to 2 us: one bf16 accumulation of 64 tiles a CTA is sure to
    # outlast it, an fp32 one of eight tiles or 32 tiles in all may not
    if dtype == torch.bfloat16 and inner == 65536:
        assert any(st == 6 for st, _ in seen), "no wait ran out"
    for _ in range(3):
        y.fill_(0)
        call()
        assert k3mx.k3mx_device_status() == (0, 0)
        assert torch.equal(y, clean)


@pytest.mark.parametrize("rows,inner,out", [(2, 16384, 12800), (64, 65536, 5120)])
def test_a_call_that_gave_up_leaves_nothing_behind(cuda_dev, rows, inner, out):
    """Calls that may give up one after another, the limit set back (which waits
    for the device), and a right one at once."""
    y, call = product(rows, inner, out, torch.float32)
    call()
    clean = y.clone()
    torch.cuda.synchronize()
    for _ in range(5):
        k3mx.k3mx_set_wait_limit(1)
        for _ in range(3):
            call()
        k3mx.k3mx_set_wait_limit(0)
        call()
        torch.cuda.synchronize()
        assert torch.equal(y, clean)
    k3mx.k3mx_device_status()
