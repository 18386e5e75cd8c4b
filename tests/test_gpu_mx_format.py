"""Microscaled formats and the quantising norm on the GPU against the
double-precision definitions.  Quantisation is exact, so codes and scales are
compared bit for bit; the norm's fp32 arithmetic is allowed 2^-20 relative
(its header's bound) before the roundings that the formats define."""
import numpy as np
import pytest
import torch

import mx_ref
import mxfp4_routed_expert_k3mx_gb300 as k3mx

pytestmark = pytest.mark.gpu
FMTS = [k3mx.K3MX_MXFP4, k3mx.K3MX_MXFP8]
BF16, F32 = torch.bfloat16, torch.float32
DELTA = 2.0 ** -20


def quantized(x, fmt):
    """(codes one per byte, scale bytes) of a device tensor, as numpy."""
    r, c = x.shape
    codes = torch.full((r, c // 2 if fmt == k3mx.K3MX_MXFP4 else c), 0xA5, dtype=torch.uint8, device=x.device)
    scales = torch.full((r, c // 32), 0xA5, dtype=torch.uint8, device=x.device)
    k3mx.k3mx_mx_quantize(codes, scales, x, fmt)
    got = codes.cpu().numpy()
    return mx_ref.unpack(got) if fmt == k3mx.K3MX_MXFP4 else got, scales.cpu().numpy(), codes, scales


def check_quantize(x, fmt):
    code, s, _, _ = quantized(x, fmt)
    rc, rs = mx_ref.quantize(x.double().cpu().numpy(), fmt)
    assert np.array_equal(s, rs)
    assert np.array_equal(code, rc)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 7168), (3, 96), (65, 1120), (300, 3584), (1025, 32)])
def test_quantize_is_exact(cuda_dev, fmt, dtype, rows, cols):
    g = torch.Generator(device=cuda_dev).manual_seed(rows * cols + fmt)
    x = torch.randn(rows, cols, generator=g, device=cuda_dev) * torch.exp(
        3.0 * torch.randn(rows, 1, generator=g, device=cuda_dev))
    check_quantize(x.to(dtype), fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad,shift", [(8, 0), (32, 8), (1, 0), (3, 1), (96, 5)])
def test_quantize_strided_and_misaligned_rows(cuda_dev, fmt, dtype, pad, shift):
    wide = torch.randn(37, 256 + pad + shift, device=cuda_dev).to(dtype)
    check_quantize(wide[:, shift:shift + 256], fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_edges(cuda_dev, fmt):
    """Ties, tops of the range, every power of two, subnormals, zeros, the
    largest fp32 values, blocks with Inf and NaN."""
    top = mx_ref.TOP[fmt]
    grid = mx_ref.GRID[fmt]
    mids = (grid[1:] + grid[:-1]) / 2
    rows = []
    for e in (-120, -20, 0, 60, 110):
        v = np.concatenate([grid, mids])
        for i in range(0, len(v), 30):
            b = np.zeros(32)
            b[0], b[1] = top, -top / 3
            b[2:2 + len(v[i:i + 30])] = v[i:i + 30] * np.where(np.arange(len(v[i:i + 30])) % 3 == 2, -1, 1)
            rows.append(b * 2.0 ** e)
    for e in range(-149, 128):                              # one value of each power of two, and its neighbours
        for f in (1.0, 1.5, 1.75, 1.5 + 2.0 ** -23, 1.75 + 2.0 ** -23, 2.0 - 2.0 ** -23):
            b = np.zeros(32)
            b[e % 32] = f * 2.0 ** e
            b[(e + 1) % 32] = -2.0 ** max(e - 1, -149)
            rows.append(b)
    rows.append(np.zeros(32))
    rows.append(np.full(32, -0.0))
    with np.errstate(all="ignore"):
        x = np.array(rows).astype(np.float32)
    for bad in (np.inf, -np.inf, np.nan):
        b = np.ones((1, 32), np.float32)
        b[0, 31] = bad
        x = np.concatenate([x, b])
    x = torch.from_numpy(x).to(cuda_dev)
    k3mx.k3mx_device_status()
    check_quantize(x, fmt)
    n = x.shape[0]
    st, row = k3mx.k3mx_device_status()
    if fmt == k3mx.K3MX_MXFP4:                              # a dropped block is reported
        assert st == 1 and n - 3 <= row < n
    else:
        assert (st, row) == (0, 0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (7, 96), (257, 1120)])
def test_dequantize_gives_the_values(cuda_dev, fmt, dtype, rows, cols):
    rng = np.random.default_rng(rows + cols)
    code = rng.integers(0, 16 if fmt == k3mx.K3MX_MXFP4 else 256, (rows, cols)).astype(np.uint8)
    s = rng.integers(0, 256, (rows, cols // 32)).astype(np.uint8)
    s.flat[0] = 255
    codes = torch.from_numpy(mx_ref.pack(code) if fmt == k3mx.K3MX_MXFP4 else code).to(cuda_dev)
    y = torch.empty(rows, cols, dtype=dtype, device=cuda_dev)
    k3mx.k3mx_mx_dequantize(y, codes, torch.from_numpy(s).to(cuda_dev), fmt)
    with np.errstate(over="ignore"):
        ref = torch.from_numpy(mx_ref.values(code, s, fmt).astype(np.float32)).to(dtype).float().numpy()
    got = y.float().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got[~np.isnan(ref)], ref[~np.isnan(ref)])


def test_round_trip_is_idempotent(cuda_dev):
    x = torch.randn(64, 512, device=cuda_dev)
    for fmt in FMTS:
        _, _, codes, scales = quantized(x, fmt)
        y = torch.empty_like(x)
        k3mx.k3mx_mx_dequantize(y, codes, scales, fmt)
        z = torch.empty_like(x)
        _, _, codes, scales = quantized(y, fmt)
        k3mx.k3mx_mx_dequantize(z, codes, scales, fmt)
        assert torch.equal(y, z)


# ------------------------------------------------------------------ norm --

def run_norm(x, r, w, eps, normed=True, inplace=False):
    t, d = x.shape
    codes = torch.full((t, d), 0xA5, dtype=torch.uint8, device=x.device)
    scales = torch.full((t, d // 32), 0xA5, dtype=torch.uint8, device=x.device)
    out = torch.full((t, d), float("nan"), dtype=BF16, device=x.device) if normed else None
    s = None if r is None else (r if inplace else torch.empty(t, d, dtype=x.dtype, device=x.device))
    k3mx.k3mx_rmsnorm_mx(codes, scales, s, x, r, w, eps, normed=out)
    return codes, scales, s, out


def check_norm(x, r, w, eps, **kw):
    s = x.double() if r is None else x.double() + r.double()
    n = (s / torch.sqrt(s.square().mean(1, keepdim=True) + eps) * w.double()).cpu().numpy()
    codes, scales, got_s, normed = run_norm(x, r, w, eps, **kw)
    if r is not None:
        assert torch.equal(got_s, (s.float()).to(x.dtype))
    if normed is not None:
        # the rounding of some value within the bound of n (rounding is monotonic)
        mag, got = torch.from_numpy(np.abs(n)), normed.double().abs().cpu()
        lo, hi = ((mag * f).to(BF16).double() for f in (1 - DELTA, 1 + DELTA))
        assert torch.all((lo <= got) & (got <= hi))
        assert torch.all((normed.double().cpu() * torch.from_numpy(n)) >= 0)
    code, sb = codes.cpu().numpy(), scales.cpu().numpy()
    m = np.abs(n).reshape(*sb.shape, 32).max(-1)
    nz = m > 0
    lo, hi = (mx_ref.scale_exponent(np.where(nz, m * f, 1.0), mx_ref.MXFP8) + 127 for f in (1 - DELTA, 1 + DELTA))
    assert np.all(np.where(nz, (lo <= sb) & (sb <= hi), sb == 0))
    e = np.exp2(sb.astype(np.float64) - 127.0).repeat(32, axis=1)
    a = np.abs(n) / e
    mag = code % 128
    assert np.all(mx_ref.nearest(mx_ref.E4M3, a * (1 - DELTA)) <= mag)
    assert np.all(mag <= mx_ref.nearest(mx_ref.E4M3, a * (1 + DELTA)))
    assert np.array_equal((code >= 128)[n != 0], (n < 0)[n != 0])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,d", [(1, 32), (1, 7168), (5, 64), (33, 1120), (257, 2048), (2, 8224), (3, 16384), (2, 32768)])
def test_norm(cuda_dev, dtype, t, d):
    g = torch.Generator(device=cuda_dev).manual_seed(t + d)
    x = torch.randn(t, d, generator=g, device=cuda_dev).to(dtype)
    r = (3 * torch.randn(t, d, generator=g, device=cuda_dev)).to(dtype)
    w = (1 + 0.2 * torch.randn(d, generator=g, device=cuda_dev)).to(BF16)
    check_norm(x, r, w, 1e-5)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_forms(cuda_dev, dtype):
    """No residual; the sum in place of the residual; strided rows; no bf16
    output; many rows; zero rows (the norm of nothing is zero)."""
    x = torch.randn(70, 512, device=cuda_dev).to(dtype)
    w = torch.randn(512, device=cuda_dev).to(BF16)
    check_norm(x, None, w, 1e-6)
    check_norm(x, x.clone(), w, 1e-6, inplace=True)
    wide = torch.randn(70, 512 + 64, device=cuda_dev).to(dtype)
    check_norm(wide[:, 32:32 + 512], x, w, 0.0, normed=False)
    z = x.clone()
    z[3] = 0
    z[69] = 0
    check_norm(z, None, w, 1e-5)
    big = torch.randn(4099, 96, device=cuda_dev).to(dtype)
    check_norm(big, big.flip(0).contiguous(), w[:96].contiguous(), 1e-5)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,d", [(700, 64), (40, 1120), (1300, 512), (20, 7168), (300, 7168), (1000, 7168), (9, 16384)])
def test_norm_codes_are_the_exact_ones(cuda_dev, dtype, t, d):
    """Sums that fp32 holds, so that only the norm rounds: its sum of squares,
    by at most fifteen roundings of 2^-24 (a thread's eight squares to a part, its
    parts' two levels, a warp's five), halved by the root: every code and scale
    is the exact norm's within 2^-20.  Those are roundings of parts and average
    out to 2^-27 and less: of codes 0.09 apart, one in several million goes the
    other way.  One in 10^6 is allowed, and of bf16 values, 0.004 apart, 20."""
    g = torch.Generator(device=cuda_dev).manual_seed(t + d)
    x = torch.randn(t, d, generator=g, device=cuda_dev)
    r = 4 * torch.randn(t, d, generator=g, device=cuda_dev)
    x, r = ((128 * v).round().clamp(-255, 255).div(128).to(dtype) for v in (x, r))
    w = (1 + 0.1 * torch.randn(d, generator=g, device=cuda_dev)).to(BF16)
    eps = 2.0 ** -17
    check_norm(x, r, w, eps, normed=False)
    codes, scales, _, normed = run_norm(x, r, w, eps)
    bare = run_norm(x, r, w, eps, normed=False)
    assert torch.equal(codes, bare[0]) and torch.equal(scales, bare[1])
    s = x.double() + r.double()
    n = (s / torch.sqrt(s.square().mean(1, keepdim=True) + eps) * w.double()).cpu().numpy()
    code, sb = mx_ref.quantize(n, mx_ref.MXFP8)
    off = np.count_nonzero(codes.cpu().numpy() != code)
    f, e = np.frexp(n)
    off16 = np.count_nonzero(normed.double().cpu().numpy() != np.ldexp(np.rint(f * 256), e - 8))
    assert np.array_equal(scales.cpu().numpy(), sb)
    assert off <= 1 + 1e-6 * n.size and off16 <= 2 + 2e-5 * n.size


def test_norm_of_nan_row_is_nan_blocks(cuda_dev):
    x = torch.randn(4, 256, device=cuda_dev)
    x[1, 7] = float("nan")
    x[2, 200] = float("inf")
    w = torch.ones(256, dtype=BF16, device=cuda_dev)
    codes, scales, _, normed = run_norm(x, None, w, 1e-5)
    # one NaN reaches every value of its row; an Inf makes its own place NaN, the others zero
    assert torch.all(scales[1] == 255) and torch.all(codes[1] == 0) and torch.isnan(normed[1]).all()
    assert scales[2, 6] == 255 and torch.isnan(normed[2, 200]) and torch.all(normed[2, :192] == 0)
    ok = [0, 3]
    ref = run_norm(x[ok].contiguous(), None, w, 1e-5)
    assert torch.equal(codes[ok], ref[0]) and torch.equal(scales[ok], ref[1])
    assert k3mx.k3mx_device_status() == (0, 0)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_past_2_31_elements(cuda_dev, fmt):
    """300 000 rows of 7200 bf16 (flat, then strided): the last rows lie past
    2^32 bytes of x and 2^31 codes."""
    rows, cols = 300_000, 7200
    wide = torch.zeros(rows, cols + 8, dtype=BF16, device=cuda_dev)
    pick = torch.tensor([0, 1, 149_130, 298_261, 298_262, rows - 1], device=cuda_dev)
    wide[pick] = torch.randn(len(pick), cols + 8, device=cuda_dev).to(BF16)
    for x in (wide[:, :cols], wide.view(-1)[:rows * cols].view(rows, cols)):
        vals = x[pick].double().cpu().numpy()
        codes = torch.empty(rows, cols // 2 if fmt == k3mx.K3MX_MXFP4 else cols, dtype=torch.uint8, device=cuda_dev)
        scales = torch.empty(rows, cols // 32, dtype=torch.uint8, device=cuda_dev)
        k3mx.k3mx_mx_quantize(codes, scales, x, fmt)
        got = codes[pick].cpu().numpy()
        rc, rs = mx_ref.quantize(vals, fmt)
        assert np.array_equal(mx_ref.unpack(got) if fmt == k3mx.K3MX_MXFP4 else got, rc)
        assert np.array_equal(scales[pick].cpu().numpy(), rs)
        y = torch.empty(rows, cols, dtype=BF16, device=cuda_dev)
        k3mx.k3mx_mx_dequantize(y, codes, scales, fmt)
        ref = torch.from_numpy(mx_ref.values(rc, rs, fmt)).to(BF16)
        assert torch.equal(y[pick].cpu(), ref)
        del codes, scales, y
