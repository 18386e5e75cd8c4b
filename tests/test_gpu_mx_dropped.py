"""Lone weight blocks of scale 255 (what the quantiser makes of a block that
holds one Inf or NaN): in a matrix of ordinary blocks they are rare, so that the
kernel meets them in a scale group whose neighbours hold none.

A dropped block adds exactly 0, as a block of zero codes under any scale does.
So y has to equal, bit for bit and in every repetition, the product with that
block's codes zero and its scale 1, which takes no such path; and that product is
compared with double precision.  Scales are all near one another: a block more or
less moves a sum of K columns by 1 / sqrt(K / 32) of it, thousands of times the
header's bound."""
import numpy as np
import pytest
import torch

import mx_ref
import mxfp4_routed_expert_k3mx_gb300 as k3mx
from test_gpu_mx_product import BF16, F32, assert_close, dev, grouped_reference

pytestmark = pytest.mark.gpu


def plain_inputs(rows, inner, shape, seed):
    rng = np.random.default_rng(seed)
    xc = rng.integers(0, 256, (rows, inner)).astype(np.uint8)
    xc[(xc & 127) == 127] = 8
    xs = rng.integers(124, 128, (rows, inner // 32)).astype(np.uint8)
    p = rng.integers(0, 256, shape + (inner // 2,)).astype(np.uint8)
    ws = rng.integers(124, 128, shape + (inner // 32,)).astype(np.uint8)
    return xc, xs, p, ws


def check(product, p, ws, blocks, repeats):
    """product(p, ws) with the blocks (index into ws) dropped, against their
    codes zero, `repeats` times."""
    zp, zs = p.clone(), ws.clone()
    dropped = ws.clone()
    for b in blocks:
        *row, k = b
        zp[tuple(row)][16 * k:16 * k + 16] = 0
        zs[tuple(row)][k] = 127
        dropped[tuple(row)][k] = 255
    want = product(zp, zs)
    for i in range(repeats):
        got = product(p, dropped)
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8)), (
            f"blocks {blocks[:4]}, repetition {i}: {(got != want).sum().item()} of {got.numel()} values differ, "
            f"in rows {(got != want).any(1).nonzero().flatten()[:8].tolist()}, "
            f"outputs {(got != want).any(0).nonzero().flatten()[:8].tolist()}")
    return want


SIZES = [(2, 7168, 300), (16, 1024, 300), (40, 7168, 300), (64, 3584, 300), (100, 7168, 300), (128, 1152, 130),
         (300, 7168, 300), (300, 1024, 130), (4096, 2048, 1000)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,inner,out", SIZES)
def test_one_block_in_each_scale_group(cuda_dev, dtype, rows, inner, out):
    """One dropped block, in turn in every group of 512 columns."""
    a = plain_inputs(rows, inner, (out,), rows + inner)
    xc, xs, p, ws = dev(*a)

    def product(p, ws):
        return k3mx.k3mx_mx_linear(torch.full((rows, out), float("nan"), dtype=dtype, device="cuda:0"), xc, xs, p, ws)

    rng = np.random.default_rng(1)
    for g in range(0, inner // 32, 16):
        block = (int(rng.integers(out)), int(min(g + rng.integers(16), inner // 32 - 1)))
        check(product, p, ws, [block], 6)
    a[3][block] = 255
    y, ad = mx_ref.product(*a)
    assert_close(check(product, p, ws, [block], 1), y, ad, dtype)
    assert k3mx.k3mx_device_status() == (0, 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,inner,out", [(2, 512, 90_000), (40, 512, 90_000), (40, 896, 60_000), (100, 512, 60_000),
                                            (300, 512, 30_000), (300, 1152, 30_000)])
def test_one_block_in_a_few_items(cuda_dev, dtype, rows, inner, out):
    """Short inner widths and many outputs, so that a CTA takes several items of
    one to three groups: dropped blocks in a random few of 128 outputs each."""
    xc, xs, p, ws = dev(*plain_inputs(rows, inner, (out,), rows + inner))

    def product(p, ws):
        return k3mx.k3mx_mx_linear(torch.full((rows, out), float("nan"), dtype=dtype, device="cuda:0"), xc, xs, p, ws)

    rng = np.random.default_rng(2)
    for part in (0.5, 0.1):
        tiles = np.flatnonzero(rng.random(out // 128) < part)
        blocks = [(int(128 * t + rng.integers(128)), int(rng.integers(inner // 32))) for t in tiles]
        check(product, p, ws, blocks, 6)
    pick = np.unique([b[0] for b in blocks[:20]] + [0, 1, out - 1])
    y, ad = mx_ref.product(*[v.cpu().numpy() for v in (xc, xs, p[pick], ws[pick])])
    assert_close(product(p, ws)[:, pick], y, ad, dtype)
    assert k3mx.k3mx_device_status() == (0, 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("counts,inner,out", [([1] * 16, 3584, 300), ([0, 40, 3, 64, 20], 3584, 300),
                                              ([0, 300, 1, 130, 40], 2048, 300), ([700, 0, 513], 1152, 1000)])
def test_one_block_a_matrix_of_a_grouped_product(cuda_dev, dtype, counts, inner, out):
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows, E = int(offsets[-1]), len(counts)
    a = plain_inputs(rows, inner, (E, out), rows + inner)
    xc, xs, p, ws, off = dev(*a, offsets)

    def product(p, ws):
        y = torch.full((rows, out), float("nan"), dtype=dtype, device="cuda:0")
        return k3mx.k3mx_mx_grouped(y, xc, xs, p, ws, off)

    rng = np.random.default_rng(3)
    for g in range(0, inner // 32, 16):
        blocks = [(e, int(rng.integers(out)), int(min(g + rng.integers(16), inner // 32 - 1)))
                  for e in range(E) if rng.random() < 0.6]
        want = check(product, p, ws, blocks, 4)
    for b in blocks:
        a[3][b] = 255
    y, ad = grouped_reference(a, offsets, out, 0.0)
    assert_close(want, y, ad, dtype)
    assert k3mx.k3mx_device_status() == (0, 0)


@pytest.mark.parametrize("rows", [3, 50, 120, 500])
def test_block_that_the_quantiser_drops(cuda_dev, rows):
    """Masters with one Inf and one NaN, quantised, multiplied: as if those two
    blocks were zero."""
    inner, out = 4096, 384
    gen = torch.Generator(device="cuda:0").manual_seed(rows)
    w = torch.randn(out, inner, generator=gen, device="cuda:0")
    x = torch.randn(rows, inner, generator=gen, device="cuda:0")
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda:0")
    c, s = k3mx.k3mx_mx_quantize(u8(rows, inner), u8(rows, inner // 32), x, k3mx.K3MX_MXFP8)

    def product(w):
        p, ws = k3mx.k3mx_mx_quantize(u8(out, inner // 2), u8(out, inner // 32), w, k3mx.K3MX_MXFP4)
        return k3mx.k3mx_mx_linear(torch.empty(rows, out, device="cuda:0"), c, s, p, ws)

    k3mx.k3mx_device_status()
    bad, zero = w.clone(), w.clone()
    bad[200, 2500], bad[17, 4000] = float("inf"), float("nan")
    zero[200, 2496:2528], zero[17, 4000:4032] = 0, 0
    want = product(zero)
    assert torch.isfinite(want).all()
    for _ in range(10):
        assert torch.equal(product(bad), want)
    st, row = k3mx.k3mx_device_status()
    assert st == 1 and row in (17, 200)
