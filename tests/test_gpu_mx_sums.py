"""What long sums lose, at its worst: the header's 4e-5 (fp32) and 3e-4 (bf16)
of sum |x w|, where those come from (an accumulation of n columns loses at most
n 2^-25 + n / 32 (2^-23 + 2^-25) of it: 3.6e-5 and 2.8e-4 for 1024 and 8192
columns; the up to 72 fp32 additions of accumulations and parts 2^-24 each, 4e-6)."""
import numpy as np
import pytest
import torch

import mx_ref
import mxfp4_routed_expert_k3mx_gb300 as k3mx
from test_gpu_mx_product import BF16, F32, dev

pytestmark = pytest.mark.gpu
BOUND = {BF16: 3e-4, F32: 4e-5}


def check(xc, xs, code, ws, rows, dtype, times=1):
    """times: how often the weights are repeated, as further outputs (with enough
    of them the inner width is not shared by the CTAs of a cluster)."""
    p = mx_ref.pack(code)
    y, ad = mx_ref.product(xc, xs, p, ws)
    got = torch.empty(rows, times * code.shape[0], dtype=dtype, device="cuda:0")
    d = dev(np.repeat(xc, rows, 0), np.repeat(xs, rows, 0), p, ws)
    k3mx.k3mx_mx_linear(got, d[0], d[1], d[2].repeat(times, 1), d[3].repeat(times, 1))
    err = np.abs(got.double().cpu().numpy().reshape(rows, times, -1) - y)
    bound = BOUND[dtype] * ad + (2.0 ** -8 * np.abs(y) if dtype == BF16 else 0)
    assert np.all(err <= bound), f"worst {np.max(err / bound):.2f} of the bound, {np.max(err / ad):.1e} of sum |x w|"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [2, 40, 100, 300])
@pytest.mark.parametrize("inner", [1024, 7168, 8192, 65536])
def test_a_large_term_before_many_small_ones(cuda_dev, rows, inner, dtype):
    """1 (or 4) first, then 2^-24 to 2^-28 of it in every column, the large term
    taken away again by the last block, so that y is what the small ones left."""
    out = 10
    code = np.full((out, inner), 2, np.uint8)                     # 1.0
    code[5:] = 3                                                  # 1.5
    ws = np.zeros((out, inner // 32), np.uint8)
    ws[:] = (127 - 24 - np.arange(out) % 5)[:, None]
    for side, sign in ((0, 0), (-1, 8)):
        ws[:, side] = 127
        block = code[:, :32] if side == 0 else code[:, -32:]
        block[:] = 0
        block[:, 0] = sign + np.where(np.arange(out) < 5, 2, 6)   # 1 or 4
    for times in (1, 960):
        check(np.full((1, inner), 0x38, np.uint8), np.full((1, inner // 32), 127, np.uint8), code, ws, rows, dtype, times)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [2, 40, 100, 300])
@pytest.mark.parametrize("inner", [1024, 7168, 65536])
def test_sums_of_one_sign(cuda_dev, rows, inner, dtype):
    """Random terms of one sign and of spread sizes, all but cancelled by the
    last 128 columns."""
    rng = np.random.default_rng(inner)
    out = 40
    xc = rng.integers(0x30, 0x48, (1, inner)).astype(np.uint8)
    xs = rng.integers(116, 120, (1, inner // 32)).astype(np.uint8)
    code = rng.integers(1, 8, (out, inner)).astype(np.uint8)
    ws = rng.integers(116, 120, (out, inner // 32)).astype(np.uint8)
    xs[:, :4], ws[:, :4], xc[:, -128:], xs[:, -4:] = 127, 127, 0x38, 127
    code[:, -128:] = 0
    y, _ = mx_ref.product(xc, xs, mx_ref.pack(code), ws)
    for n in range(out):
        rest = y[0, n]
        top = int(np.ceil(np.log2(rest / (32 * 6))))
        for b in range(4):
            ws[n, -4 + b] = 127 + top - 5 * b
            for i in range(32):
                k = int(np.searchsorted(mx_ref.E2M1, rest / 2.0 ** (top - 5 * b), side="right")) - 1
                code[n, inner - 128 + 32 * b + i] = 8 + k
                rest -= mx_ref.E2M1[k] * 2.0 ** (top - 5 * b)
    check(xc, xs, code, ws, rows, dtype)
