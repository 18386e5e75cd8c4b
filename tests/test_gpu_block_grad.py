"""The activation with its inputs saved in 8 bits, and the backward passes that
read what was saved, against the double-precision definitions."""
import numpy as np
import pytest
import torch

import block_ref
import mx_ref
import mxfp4_routed_expert_k3mx_gb300 as k3mx

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16}


def u8(*shape):
    return torch.full(shape, 0x5A, dtype=torch.uint8, device=DEV)


def doubles(t):
    return t.detach().cpu().double().numpy()


def rows_of(x, kind, pad):
    wide = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=TYPES[kind], device=DEV)
    wide[:, :x.shape[1]] = torch.from_numpy(x).to(DEV).to(TYPES[kind])
    return wide[:, :x.shape[1]]


def situ(gu, save):
    R, F = gu.shape[0], gu.shape[1] // 2
    out = [u8(R, F), u8(R, F // 32)] + ([u8(R, 2 * F), u8(R, 2 * F // 32)] if save else [None, None])
    k3mx.k3mx_situ_mx(out[0], out[1], gu, saved=out[2], saved_scales=out[3])
    return out


def off_of_h(g, u):
    """What the gradients' factors may be off by, relative."""
    return 2.0 ** -18 * (1 + (np.abs(g) + np.abs(u)) / 16)


SHAPES = [(1, 32), (1, 2048), (3, 96), (16, 2048), (37, 1056), (300, 256), (1000, 32), (129, 4096)]


@pytest.mark.parametrize("R,F", SHAPES)
@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("pad", [0, 40])
def test_situ(cuda_dev, R, F, kind, pad):
    r = np.random.default_rng(R + F)
    x = r.normal(size=(R, 2 * F)) * np.exp(r.normal(size=2 * F))
    x[:, r.integers(0, 2 * F, 3)] *= 30
    gu = rows_of(x, kind, pad)
    codes, scales, saved, ss = situ(gu, True)
    x = doubles(gu)
    code, s = mx_ref.quantize(x, mx_ref.MXFP8)
    assert np.array_equal(saved.cpu().numpy(), code) and np.array_equal(ss.cpu().numpy(), s)
    g, u = x[:, :F], x[:, F:]
    h = block_ref.situ(g, u)
    # h's own codes (values near a middle are formed within 2^-29: one in 30 million may still turn); below g = -16 a neighbour's
    want, s = mx_ref.quantize(h, mx_ref.MXFP8)
    got = codes.cpu().numpy()
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(got[g >= -16], want[g >= -16]) and np.abs((got & 127).astype(int) - (want & 127)).max() <= 1
    alone = situ(gu, False)
    assert torch.equal(alone[0], codes) and torch.equal(alone[1], scales)
    assert k3mx.k3mx_device_status() == (0, 0)


def test_situ_of_extreme_values(cuda_dev):
    inf, nan = float("inf"), float("nan")
    g = np.zeros((1, 7 * 32))
    u = np.ones_like(g) * 25.0
    g[0, :32], g[0, 32:64] = inf, -inf
    g[0, 64], g[0, 96:128] = nan, 3e38
    g[0, 128:160], u[0, 160:192], u[0, 192:] = -3e38, inf, -inf
    g[0, 160:] = 4.0
    gu = rows_of(np.concatenate([g, u], 1), "float32", 0)
    codes, scales, saved, ss = situ(gu, True)
    got = mx_ref.values(codes.cpu().numpy(), scales.cpu().numpy(), mx_ref.MXFP8)[0]
    top = 100 * np.tanh(1.0)
    close = lambda v, want: np.all(np.abs(v - want) <= 2.0 ** -4 * abs(want))
    assert close(got[:32], top) and np.all(got[32:64] == 0) and np.all(np.isnan(got[64:96])) and close(got[96:128], top)
    assert np.all(got[128:160] == 0)
    s4 = 4 * np.tanh(1.0) / (1 + np.exp(-4.0)) * 25
    assert close(got[160:192], s4) and close(got[192:], -s4)
    assert np.array_equal(ss.cpu().numpy()[0], np.where(np.isin(np.arange(14), [0, 1, 2, 12, 13]), 255, ss.cpu().numpy()[0]))
    assert not np.any(ss.cpu().numpy()[0][[3, 4, 5, 6, 7, 8, 9, 10, 11]] == 255)
    dgu = torch.empty(1, 14 * 32, device=DEV)
    k3mx.k3mx_situ_mx_backward(dgu, torch.ones(1, 7 * 32, device=DEV), saved, ss)
    bad = np.isnan(doubles(dgu)[0]).reshape(2, 7, 32)
    assert np.all(bad[:, [0, 1, 2, 5, 6]]) and not np.any(bad[:, [3, 4]])
    assert np.all(doubles(dgu)[0].reshape(2, 7, 32)[0, 3:5] == 0) and k3mx.k3mx_device_status() == (0, 0)


@pytest.mark.parametrize("kind", sorted(TYPES))
def test_situ_where_one_factor_is_a_limit(cuda_dev, kind):
    """h = 4 b(u) and 25 a(g), of many values: some are near the middle of two codes."""
    r = np.random.default_rng(7)
    for other in (1.0, -1.0):
        x = np.concatenate([np.full((512, 256), np.inf), r.normal(size=(512, 256)) * 8], 1)
        for gate in (True, False):
            if not gate:
                x = np.concatenate([x[:, 256:], other * x[:, :256]], 1)
            gu = rows_of(x, kind, 0)
            codes, scales, _, _ = situ(gu, False)
            g, u = doubles(gu)[:, :256], doubles(gu)[:, 256:]
            want, s = mx_ref.quantize(block_ref.situ(np.minimum(g, 1e3), np.clip(u, -1e4, 1e4)), mx_ref.MXFP8)
            got = codes.cpu().numpy()
            assert np.array_equal(scales.cpu().numpy(), s)
            assert np.array_equal(got[g >= -16], want[g >= -16])


@pytest.mark.parametrize("save", [False, True])
def test_situ_of_many_rows(cuda_dev, save):
    """Every bf16 value of g with some of u and the other way round, in a call of
    many rows and in calls of few."""
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    r = np.random.default_rng(8)
    R, F = 16640, 512                                             # (1 M runs and more)
    x = torch.from_numpy(r.normal(size=(R, 2 * F)) * np.exp(r.normal(size=(1, 2 * F)))).bfloat16()
    finite = every[torch.isfinite(every.float())]
    n = finite.numel() // 32 * 32
    x[:n // 32, :32] = finite[:n].view(-1, 32)                     # g
    x[:n // 32, F + 32:F + 64] = finite[:n].view(-1, 32)           # u
    x[4000:4128, :F] = every.view(128, 512)
    x[5000:5128, F:] = every.view(128, 512)
    x[6000:6500] = 0
    x[6500:7000, ::3] = 0
    x[7000:9000, 64:72] *= 300                                     # outliers beside ordinary values
    gu = x.to(DEV)
    out = situ(gu, save)
    v = doubles(gu)
    g, u = v[:, :F], v[:, F:]
    with np.errstate(all="ignore"):
        h = np.where(np.isnan(g) | np.isnan(u), np.nan, block_ref.situ(np.clip(g, -700, 1e3), np.clip(u, -1e4, 1e4)))
        # blocks whose largest is next to nothing, or has g < -16 (there codes may be others')
        m, low = np.abs(np.nan_to_num(h)).reshape(R, F // 32, 32), (g < -16).reshape(R, F // 32, 32)
        top = np.where(low, 0, m).max(-1)
        dim = (top < 2.0 ** -90) | (top < m.max(-1))
    want, s = mx_ref.quantize(np.where(np.isnan(h), np.nan, h), mx_ref.MXFP8)
    got = out[0].cpu().numpy()
    assert np.array_equal(out[1].cpu().numpy()[~dim], s[~dim])
    assert np.array_equal(out[1].cpu().numpy() == 255, s == 255)
    bright = ~dim.repeat(32, 1).reshape(R, F)
    assert np.abs((got & 127).astype(int) - (want & 127))[bright].max() <= 1
    bright &= ~low.reshape(R, F)
    assert np.array_equal(got[bright], want[bright])
    for at in (slice(0, 4200), slice(5000, 5200), slice(6000, 7100), slice(16000, R)):
        few = situ(gu[at].contiguous(), save)
        assert np.array_equal(few[1].cpu().numpy()[~dim[at]], s[at][~dim[at]])
        assert np.array_equal(few[0].cpu().numpy()[bright[at]], got[at][bright[at]])
        assert not save or (torch.equal(few[2], out[2][at]) and torch.equal(few[3], out[3][at]))
    if save:
        code, s = mx_ref.quantize(v, mx_ref.MXFP8)
        assert np.array_equal(out[2].cpu().numpy(), code) and np.array_equal(out[3].cpu().numpy(), s)
    assert k3mx.k3mx_device_status() == (0, 0)


def test_situ_of_tiny_and_zero_blocks(cuda_dev):
    x = np.zeros((3, 128))
    x[1] = 1e-38
    x[2, :64], x[2, 64:] = 1e-20, 1e-18
    codes, scales, saved, ss = situ(rows_of(x, "float32", 0), True)
    assert torch.all(codes[:2] & 127 == 0) and torch.all(scales[:2] == 0) and torch.all(ss[0] == 0)
    got = mx_ref.values(codes.cpu().numpy(), scales.cpu().numpy(), mx_ref.MXFP8)[2]
    want = block_ref.situ(np.float64(np.float32(1e-20)), np.float64(np.float32(1e-18)))      # about 5e-39: subnormal
    assert np.all(np.abs(got - want) <= 2.0 ** -4 * want + 2.0 ** -137)


@pytest.mark.parametrize("R,F", SHAPES)
@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("pad", [0, 24])
def test_situ_backward(cuda_dev, R, F, kind, pad):
    r = np.random.default_rng(R * F)
    x = r.normal(size=(R, 2 * F)) * np.exp(r.normal(size=2 * F))
    x[:, r.integers(0, 2 * F, 3)] *= 30
    code, s = mx_ref.quantize(x.astype(np.float32).astype(np.float64), mx_ref.MXFP8)
    dh = rows_of(r.normal(size=(R, F)) * 1e-3, kind, pad)
    dgu = torch.full((R, 2 * F), float("nan"), dtype=TYPES[kind], device=DEV)
    k3mx.k3mx_situ_mx_backward(dgu, dh, torch.from_numpy(code).to(DEV), torch.from_numpy(s).to(DEV))
    v = mx_ref.values(code, s, mx_ref.MXFP8)
    g, u = v[:, :F], v[:, F:]
    dg, du, mag = block_ref.situ_backward(g, u, doubles(dh))
    off = off_of_h(g, u)
    for got, want, m in ((doubles(dgu)[:, :F], dg, mag), (doubles(dgu)[:, F:], du, np.abs(du))):
        tol = off * m
        tol += block_ref.HALF[kind] * (np.abs(want) + tol) + 2.0 ** -130
        assert np.all(np.abs(got - want) <= tol)
    assert k3mx.k3mx_device_status() == (0, 0)


def test_situ_backward_is_situs_difference(cuda_dev):
    """From what the forward pass saved: h(g + d) - h(g - d) over values that 8
    bits hold exactly, in fp64 of the definition."""
    r = np.random.default_rng(1)
    x = r.integers(-15, 16, size=(4, 256)) / 4.0                    # within 4 bits of a block's largest
    gu = rows_of(x, "float32", 0)
    codes, scales, saved, ss = situ(gu, True)
    assert np.array_equal(mx_ref.values(saved.cpu().numpy(), ss.cpu().numpy(), mx_ref.MXFP8), x)
    dgu = torch.empty(4, 256, device=DEV)
    k3mx.k3mx_situ_mx_backward(dgu, torch.ones(4, 128, device=DEV), saved, ss)
    g, u, d = x[:, :128], x[:, 128:], 1e-4
    dg = (block_ref.situ(g + d, u) - block_ref.situ(g - d, u)) / (2 * d)
    du = (block_ref.situ(g, u + d) - block_ref.situ(g, u - d)) / (2 * d)
    # differences are off by d^2 / 6 of a third derivative (below 20), and by 2^-52 of h over d; the kernel by 2^-17 of two terms
    tol = 20 * d * d + 2.0 ** -52 * 100 / d
    assert np.all(np.abs(doubles(dgu) - np.concatenate([dg, du], 1)) <= tol + 2.0 ** -17 * 60)


@pytest.mark.parametrize("kind", sorted(TYPES))
def test_situ_backward_of_many_rows(cuda_dev, kind):
    """Every code under every scale, in calls of many rows and of few: the same bits, and the definition's."""
    r = np.random.default_rng(2)
    R, F = 8300, 512
    code = r.integers(0, 256, size=(R, 2 * F)).astype(np.uint8)
    s = r.integers(90, 140, size=(R, 2 * F // 32)).astype(np.uint8)
    s[:64] = r.integers(112, 127, size=(64, 2 * F // 32))
    s[64:320] = np.arange(256)[:, None]
    code[64:320] &= 0xBF                                # (smaller values: no infinity below scale 254)
    dh = rows_of(r.normal(size=(R, F)), kind, 8)
    dev = lambda t: torch.from_numpy(t).to(DEV)
    dgu = torch.full((R, 2 * F), 99.0, dtype=TYPES[kind], device=DEV)
    k3mx.k3mx_situ_mx_backward(dgu, dh, dev(code), dev(s))
    for at in (slice(0, 64), slice(64, 320), slice(8000, 8300)):
        few = torch.empty(at.stop - at.start, 2 * F, dtype=TYPES[kind], device=DEV)
        k3mx.k3mx_situ_mx_backward(few, dh[at], dev(code[at]), dev(s[at]))
        assert torch.equal(few.nan_to_num(12345.0, 1e38, -1e38), dgu[at].nan_to_num(12345.0, 1e38, -1e38))
    v = mx_ref.values(code, s, mx_ref.MXFP8)
    bad = np.isnan(v[:, :F]) | np.isnan(v[:, F:])
    got = doubles(dgu)
    assert np.all(np.isnan(got[:, :F]) == bad) and np.all(np.isnan(got[:, F:]) == bad)
    big = (np.abs(v) > 1e30)[:, :F] | (np.abs(v) > 1e30)[:, F:]
    v = np.where(np.isnan(v) | (np.abs(v) > 1e30), 0.0, v)
    g, u = v[:, :F], v[:, F:]
    dg, du, mag = block_ref.situ_backward(g, u, doubles(dh))
    off = off_of_h(g, u)
    for have, want, m in ((got[:, :F], dg, mag), (got[:, F:], du, np.abs(du))):
        # exponentials below 2^-126 are taken for 0: 4 * 25 of them, below 2^7, are dg's and du's
        tol = off * m + 2.0 ** -119 * np.abs(doubles(dh))
        tol += block_ref.HALF[kind] * (np.abs(want) + tol) + 2.0 ** -120
        assert np.all((np.abs(have - want) <= tol) | bad | big)


# --------------------------------------------------------------- the norm --

def norm_backward(x, dn, weight, eps, dres, kind, pad=0, into_dres=False):
    """x: doubles [T, W] quantised here; returns (dx, dweight) and the definition's results."""
    T, W = x.shape
    code, s = mx_ref.quantize(x.astype(np.float32).astype(np.float64), mx_ref.MXFP8)
    dn, g = rows_of(dn, kind, pad), torch.from_numpy(weight).to(DEV).bfloat16()
    res = None if dres is None else rows_of(dres, kind, 0).contiguous()
    want = block_ref.norm_backward(mx_ref.values(code, s, mx_ref.MXFP8), doubles(dn), doubles(g), np.float64(np.float32(eps)),
                                   None if res is None else doubles(res))
    dx = res if into_dres else torch.full((T, W), float("nan"), dtype=TYPES[kind], device=DEV)
    dweight = torch.full((W,), float("nan"), device=DEV)
    ws = torch.full((k3mx.k3mx_rmsnorm_mx_backward_workspace_size(T, W) // 4,), float("nan"), device=DEV)
    k3mx.k3mx_rmsnorm_mx_backward(dx, dweight, dn, torch.from_numpy(code).to(DEV), torch.from_numpy(s).to(DEV), g, eps, ws, dres=res)
    return dx, dweight, want


def check_norm(dx, dweight, want, kind, T, W):
    wx, wg, mx, mg = want
    # sums of W terms, at most W / 1024 + 32 in turn; the factor k, the products: 30 more, each half a step
    c = (W / 1024 + 32 + 30) * 2.0 ** -24
    tol = c * mx
    tol += block_ref.HALF[kind] * (np.abs(wx) + tol) + 1e-40
    assert np.all(np.abs(doubles(dx) - wx) <= tol)
    # a thread's rows, at most T / 600 + 8 of them or 1024, then the parts, each warp's 76 or T / 8192 and eight warps
    rows = min(T / 600 + 8, 1024) + max(76, T / 8192) + 16
    assert np.all(np.abs(doubles(dweight) - wg) <= (rows + W / 1024 + 40) * 2.0 ** -24 * mg + 1e-40)


@pytest.mark.parametrize("T,W", [(1, 32), (1, 7168), (2, 7168), (2, 16416), (16, 128), (17, 1024), (3, 64), (8, 256), (9, 288), (64, 1024), (65, 1056), (700, 160), (613, 2048),
                                 (200, 7168), (33, 8224), (7, 16384), (5, 16416), (3, 32768), (5000, 96), (2500, 1536)])
@pytest.mark.parametrize("kind", sorted(TYPES))
def test_norm_backward(cuda_dev, T, W, kind):
    r = np.random.default_rng(T + W)
    x = r.normal(size=(T, W)) * np.exp(r.normal(size=(1, W))) * np.exp(2 * r.normal(size=(T, 1)))
    dn, dres = r.normal(size=(T, W)) * 1e-3 * np.exp(r.normal(size=(T, 1))), r.normal(size=(T, W)) * 1e-3
    w = 1 + 0.1 * r.normal(size=W)
    a = norm_backward(x, dn, w, 1e-5, dres, kind)
    check_norm(*a, kind, T, W)
    b = norm_backward(x, dn, w, 1e-5, dres, kind, pad=16, into_dres=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check_norm(*norm_backward(x, dn, w, 0.5, None, kind), kind, T, W)
    assert k3mx.k3mx_device_status() == (0, 0)


@pytest.mark.parametrize("T,W", [(1 << 21, 32), (200_000, 1056)])
def test_norm_backward_of_very_many_rows(cuda_dev, T, W):
    gen = torch.Generator(device=DEV).manual_seed(4)
    saved = torch.randint(0, 0x78, (T, W), generator=gen, device=DEV, dtype=torch.uint8)
    ss = torch.randint(118, 122, (T, W // 32), generator=gen, device=DEV, dtype=torch.uint8)
    dn, g = torch.randn(T, W, generator=gen, device=DEV) + 0.5, torch.ones(W, device=DEV).bfloat16()
    dx, dw = torch.empty(T, W, device=DEV), torch.empty(W, device=DEV)
    ws = u8(k3mx.k3mx_rmsnorm_mx_backward_workspace_size(T, W))
    k3mx.k3mx_rmsnorm_mx_backward(dx, dw, dn, saved, ss, g, 1e-5, ws)
    x = saved.view(torch.float8_e4m3fn).double().view(T, W // 32, 32) * torch.exp2(ss.double() - 127)[..., None]
    x = x.view(T, W)
    n = x / torch.sqrt(x.square().mean(1, keepdim=True) + 1e-5)
    want, mag = (dn.double() * n).sum(0), (dn.double() * n).abs().sum(0)
    # 1024 rows in turn at most, then 2048 parts by 32 warps, 64 in turn, and those
    assert torch.all((dw - want).abs() <= (1024 + 64 + 32 + 40) * 2.0 ** -24 * mag)
    at = torch.tensor([0, 1, T // 2, T - 1], device=DEV)
    a, q = dn[at].double(), (dn[at].double() * n[at]).mean(1, keepdim=True)
    k = 1 / torch.sqrt(x[at].square().mean(1, keepdim=True) + 1e-5)
    assert torch.all((dx[at] - k * (a - n[at] * q)).abs() <= 100 * 2.0 ** -24 * k * (a.abs() + n[at].abs() * (a * n[at]).abs().mean(1, keepdim=True)))


def test_norm_backward_with_the_forward_pass(cuda_dev):
    """k3mx_rmsnorm_mx's own sum, saved in 8 bits, and its differences (fp64 of
    the definition) at what was saved."""
    T, W = 5, 96
    gen = torch.Generator(device=DEV).manual_seed(0)
    x, res = (torch.randn(T, W, generator=gen, device=DEV) for _ in range(2))
    g = (1 + 0.1 * torch.randn(W, generator=gen, device=DEV)).bfloat16()
    total = torch.empty_like(x)
    k3mx.k3mx_rmsnorm_mx(u8(T, W), u8(T, W // 32), total, x, res, g, 1e-5)
    saved, ss, back = u8(T, W), u8(T, W // 32), torch.empty_like(x)
    k3mx.k3mx_mx_quantize(saved, ss, total, k3mx.K3MX_MXFP8)
    k3mx.k3mx_mx_dequantize(back, saved, ss, k3mx.K3MX_MXFP8)
    dn, dx, dw = torch.randn(T, W, generator=gen, device=DEV), torch.empty_like(x), torch.empty(W, device=DEV)
    ws = u8(k3mx.k3mx_rmsnorm_mx_backward_workspace_size(T, W))
    k3mx.k3mx_rmsnorm_mx_backward(dx, dw, dn, saved, ss, g, 1e-5, ws)
    f = lambda s, g: (s * g / np.sqrt((s * s).mean(1, keepdims=True) + np.float64(np.float32(1e-5))) * doubles(dn)).sum()
    s, gd, h = doubles(back), doubles(g), 1e-5
    for j in range(0, W, 7):
        e = np.zeros((T, W))
        e[2, j] = h
        # a difference is off by h^2 of a third derivative (some tens) and by 2^-52 |f| / h; the kernel by 2^-17 of terms below 20
        assert abs((f(s + e, gd) - f(s - e, gd)) / (2 * h) - doubles(dx)[2, j]) <= 1e-7 + 2.0 ** -17 * 20
        assert abs((f(s, gd + e[2]) - f(s, gd - e[2])) / (2 * h) - doubles(dw)[j]) <= 1e-7 + 2.0 ** -17 * 20


@pytest.mark.parametrize("scale", [1e18, 1e30, 1e-15])
@pytest.mark.parametrize("W", [96, 2048])
def test_norm_backward_of_large_and_small_rows(cuda_dev, scale, W):
    """Squares that leave fp32, or nearly vanish beside eps."""
    r = np.random.default_rng(3)
    x, dn = r.normal(size=(4, W)) * scale, r.normal(size=(4, W))
    check_norm(*norm_backward(x, dn, np.ones(W), 1e-20, None, "float32"), "float32", 4, W)


def test_norm_backward_of_rows_without_a_norm(cuda_dev):
    x = np.zeros((3, 64))
    x[2] = 1.0
    dn = np.ones((3, 64))
    dx, dw, want = norm_backward(x, dn, np.ones(64), 1e-5, None, "float32")
    check_norm(dx, dw, want, "float32", 3, 64)                       # zeros with eps: dx = g dn / sqrt(eps)
    with np.errstate(all="ignore"):
        dx, dw, _ = norm_backward(x, dn, np.ones(64), 0.0, None, "float32")
    assert torch.all(dx[:2].isnan()) and torch.all(dx[2].abs() < 1e-5)
    x[0, 3] = np.inf
    with np.errstate(all="ignore"):
        dx, dw, _ = norm_backward(x, dn, np.ones(64), 1e-5, None, "float32")
    assert torch.all(dx[0].isnan()) and not dx[1:].isnan().any() and torch.all(dw.isnan())


def test_pitches_past_32_bits(cuda_dev):
    ld = (1 << 31) + 8
    wide = torch.empty(2 * ld + 512, dtype=torch.bfloat16, device=DEV)
    far = lambda cols: wide.as_strided((3, cols), (ld, 1))
    r = np.random.default_rng(0)
    gu = rows_of(r.normal(size=(3, 512)), "bfloat16", 0)
    far(512).copy_(gu)
    a, b = situ(far(512), True), situ(gu, True)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    out = [torch.empty(3, 512, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for o, dh in zip(out, (far(256), gu[:, :256].contiguous())):
        k3mx.k3mx_situ_mx_backward(o, dh, a[2], a[3])
    assert torch.equal(*out)
    res = []
    for dn in (far(512), gu):
        dx, dw = torch.empty(3, 512, dtype=torch.bfloat16, device=DEV), torch.empty(512, device=DEV)
        k3mx.k3mx_rmsnorm_mx_backward(dx, dw, dn, a[2], a[3], torch.ones(512, device=DEV).bfloat16(), 1e-5,
                                      u8(k3mx.k3mx_rmsnorm_mx_backward_workspace_size(3, 512)))
        res.append((dx, dw))
    assert all(torch.equal(p, q) for p, q in zip(*res))


def test_elements_past_32_bits(cuda_dev):
    """dgu's last rows lie 2^32 elements behind its first."""
    R, F = (1 << 21) + 3, 1024
    saved, ss = torch.empty(R, 2 * F, dtype=torch.uint8, device=DEV), torch.empty(R, 2 * F // 32, dtype=torch.uint8, device=DEV)
    gu = torch.zeros(R, 2 * F, dtype=torch.bfloat16, device=DEV)
    gu[-2:] = torch.randn(2, 2 * F, device=DEV).bfloat16()
    codes, scales = torch.empty(R, F, dtype=torch.uint8, device=DEV), torch.empty(R, F // 32, dtype=torch.uint8, device=DEV)
    k3mx.k3mx_situ_mx(codes, scales, gu, saved=saved, saved_scales=ss)
    few = situ(gu[-2:].contiguous(), True)
    assert torch.equal(codes[-2:], few[0]) and torch.equal(scales[-2:], few[1]) and torch.equal(saved[-2:], few[2])
    assert torch.equal(ss[-2:], few[3]) and torch.all(codes[:5] == 0)
    dh = torch.ones(R, F, dtype=torch.bfloat16, device=DEV)
    k3mx.k3mx_situ_mx_backward(gu, dh, saved, ss)
    want = torch.empty(2, 2 * F, dtype=torch.bfloat16, device=DEV)
    k3mx.k3mx_situ_mx_backward(want, dh[-2:].contiguous(), few[2], few[3])
    assert torch.equal(gu[-2:], want) and torch.all(gu[:5] == 0)
