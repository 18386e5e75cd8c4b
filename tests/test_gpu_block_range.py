"""The activation and the norm's gradient at the ends of their inputs' range,
against the double-precision definitions."""
import numpy as np
import pytest
import torch

import block_ref
import mx_ref
import mxfp4_routed_expert_k3mx_gb300 as k3mx
from test_gpu_block_grad import TYPES, doubles, rows_of, situ

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF, NAN = float("inf"), float("nan")


def situ_of(g, u):
    """h in doubles, with its limits."""
    with np.errstate(all="ignore"):
        return np.where(np.isnan(g) | np.isnan(u), np.nan, block_ref.situ(np.clip(g, -700, 1e3), np.clip(u, -1e4, 1e4)))


# ---------------------------------------------------------- the activation --

GATES = [INF, 3e38, 1000, 130, 30, 1, 2.0 ** -20, 0.0, -0.0, -2.0 ** -20, -1, -16, -40, -86, -87, -88, -89, -100, -110, -111, -128,
         -128.5, -129, -130, -131, -200, -250, -300, -1000, -3e38, -INF, NAN]
UPS = [INF, 3e38, 1000, 512, 250, 25, 1, 0.0, -0.0, -1, -25, -230, -239, -240, -249, -250, -251, -256, -286, -288, -290, -300, -512, -700,
       -1000, -3e38, -INF, NAN]


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("many", [False, True])
def test_situ_of_every_extreme_with_every_other(cuda_dev, kind, many):
    """Whole blocks of one pair of values, and single pairs beside ordinary ones."""
    r = np.random.default_rng(11)
    g, u = (v.reshape(-1) for v in np.meshgrid(GATES, UPS, indexing="ij"))
    n = g.size                                               # 896 pairs: 28 blocks of each of 32 rows
    whole = [np.repeat(v.reshape(32, 28), 32, axis=1) for v in (g, u)]
    beside = [r.normal(size=(32, 896)) * 3 for _ in range(2)]
    at = r.integers(0, 32, size=n).reshape(32, 28) + 32 * np.arange(28)
    for v, w in zip(beside, (g, u)):
        np.put_along_axis(v, at, w.reshape(32, 28), axis=1)
    x = np.concatenate([np.concatenate(whole, 1), np.concatenate(beside, 1)])
    if many:                                                 # (1 M runs and more of bf16 take another form)
        x = np.concatenate([x, r.normal(size=(9400 - 64, 2 * 896)).astype(np.float32)])
    gu = rows_of(x, kind, 8)
    codes, scales, _, _ = situ(gu, False)
    v = doubles(gu)[:64]
    g, u = v[:, :896], v[:, 896:]
    h = situ_of(g, u)
    want, s = mx_ref.quantize(h, mx_ref.MXFP8)
    got, gs = codes.cpu().numpy()[:64], scales.cpu().numpy()[:64]
    assert np.array_equal(gs == 255, np.isnan(h).reshape(64, 28, 32).any(-1))
    # values: a code's half step, 2^-15 below g = -16, and 100 e^-87 where h may be taken for 0; half the smallest
    # code's step of the block
    top = np.nanmax(np.abs(np.where(np.isnan(h), 0.0, h)).reshape(64, 28, 32), -1).repeat(32, 1)
    live = ~(gs == 255).repeat(32, 1)
    val = mx_ref.values(got, gs, mx_ref.MXFP8)
    tol = (2.0 ** -4 + 2.0 ** -14) * np.abs(h) + 2.0 ** -17 * top + 2.0 ** -118
    assert np.all(np.abs(val - h)[live] <= tol[live])
    # h's own codes under its own scale, unless the block's largest is one of those
    mag, low = np.abs(h).reshape(64, 28, 32), (g < -16).reshape(64, 28, 32)
    top = np.where(low, 0.0, mag).max(-1)
    bright = (top >= 2.0 ** -90) & (top >= mag.max(-1))
    assert np.array_equal(gs[bright], s[bright])
    exact = bright.repeat(32, 1) & ~(g < -16)
    assert np.array_equal(got[exact], want[exact])
    assert k3mx.k3mx_device_status() == (0, 0)


def gates_at_a_middle():
    """fp32 gates with |25 a(g)| beyond the middle of two codes by less than 1 - tanh(10) of it, and by more
    than h is formed to."""
    def a(g):
        return 4 * np.tanh(g / 4) / (1 + np.exp(-g))
    found = []
    for lo, hi in ((2.0 ** -24, 40.0), (-1.8, -2.0 ** -24), (-16.0, -3.2)):
        steps = np.sort(np.float32(np.sign(lo) * np.exp(np.linspace(np.log(min(abs(lo), abs(hi))), np.log(max(abs(lo), abs(hi))), 8000))))
        v = np.abs(25 * a(steps.astype(np.float64)))
        for i in range(len(steps) - 1):
            e = np.floor(np.log2(min(v[i], v[i + 1])))
            for m in (np.arange(8, 16) + 0.5) * 2.0 ** (e - 3):
                if not min(v[i], v[i + 1]) < m < max(v[i], v[i + 1]):
                    continue
                l, h = np.float32(steps[i]), np.float32(steps[i + 1])          # |25 a| - m changes its sign between the two
                up = v[i + 1] > v[i]
                for _ in range(60):
                    c = np.float32((np.float64(l) + np.float64(h)) / 2)
                    if c == l or c == h:
                        break
                    if (abs(25 * a(np.float64(c))) > m) == up:
                        h = c
                    else:
                        l = c
                g = h if up else l                                             # the one beyond m
                over = abs(25 * a(np.float64(g))) / m - 1
                if 2.0 ** -28.8 < over < 2.0 ** -27.95:
                    found.append(g)
    return np.array(found, np.float64)


@pytest.mark.parametrize("u", [-INF, -1000.0, -600.0, 600.0, INF])
def test_situ_where_the_other_factor_is_next_to_its_limit(cuda_dev, u):
    g = gates_at_a_middle()
    assert g.size >= 3
    x = np.concatenate([np.repeat(g[:, None], 32, 1), np.full((g.size, 32), u)], 1)
    codes, scales, _, _ = situ(rows_of(x, "float32", 0), False)
    want, s = mx_ref.quantize(situ_of(x[:, :32], x[:, 32:]), mx_ref.MXFP8)
    assert np.array_equal(scales.cpu().numpy(), s) and np.array_equal(codes.cpu().numpy(), want)


# ---------------------------------------------------------------- the norm --

def norm_backward(x, dn, weight, eps, kind):
    """(dx, dweight) at the rows of doubles x [T, W] quantised here, and the definition's results."""
    T, W = x.shape
    code, s = mx_ref.quantize(x.astype(np.float32).astype(np.float64), mx_ref.MXFP8)
    dn, g = rows_of(dn, kind, 0).contiguous(), torch.from_numpy(weight).to(DEV).bfloat16()
    with np.errstate(all="ignore"):
        want = block_ref.norm_backward(mx_ref.values(code, s, mx_ref.MXFP8), doubles(dn), doubles(g), np.float64(np.float32(eps)), None)
    dx, dweight = torch.full((T, W), NAN, dtype=TYPES[kind], device=DEV), torch.full((W,), NAN, device=DEV)
    ws = torch.full((k3mx.k3mx_rmsnorm_mx_backward_workspace_size(T, W),), 0xFF, dtype=torch.uint8, device=DEV)
    k3mx.k3mx_rmsnorm_mx_backward(dx, dweight, dn, torch.from_numpy(code).to(DEV), torch.from_numpy(s).to(DEV), g, eps, ws)
    return dx, dweight, want


def check_norm(dx, dweight, want, kind, T, W):
    """What is off, beside fp32's own range: each sum's terms in turn and 30 roundings more."""
    wx, wg, mx, mg = want
    tol = (W / 1024 + 32 + 30) * 2.0 ** -24 * mx
    tol += block_ref.HALF[kind] * (np.abs(wx) + tol) + 2.0 ** -117
    # rows whose terms fp32 holds
    held = np.nan_to_num(mx, nan=np.inf).max(1) < 2.0 ** 127
    got = doubles(dx)
    assert np.all(np.abs(got - wx)[held] <= tol[held])
    if np.isfinite(mg).all() and mg.max() < 2.0 ** 127:
        rows = min(T / 600 + 8, 1024) + max(76, T / 8192) + 16
        assert np.all(np.abs(doubles(dweight) - wg) <= (rows + W / 1024 + 40) * 2.0 ** -24 * mg + 2.0 ** -117)
    return held


def rows_of_sizes(T, W, kind, sizes, size, eps):
    """Rows of each size and gradients of one, whose products add up or cancel."""
    r = np.random.default_rng(5)
    scale = np.resize(np.array(sizes), T)[:, None]
    unit = r.normal(size=(T, W))
    dn = np.abs(r.normal(size=(T, W))) * size
    along = (np.arange(T) // len(sizes) % 2 == 0)[:, None]
    dn = np.where(along, dn * np.sign(unit), dn * r.choice([-1.0, 1.0], size=(T, W)))
    held = check_norm(*norm_backward(unit * scale, dn, 1 + 0.1 * r.normal(size=W), eps, kind), kind, T, W)
    assert held[scale[:, 0] >= 1.0].all() and k3mx.k3mx_device_status() == (0, 0)


NORM_SHAPES = [(24, 96), (24, 2048), (168, 2048), (24, 7168), (24, 8224), (24, 16416)]


@pytest.mark.parametrize("T,W", NORM_SHAPES)
@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("size", [1.0, 1e20, 3e35, 1e36])
@pytest.mark.parametrize("eps", [0.0, 1e-5])
def test_norm_backward_of_large_gradients(cuda_dev, T, W, kind, size, eps):
    """Sums of squares and of products that leave fp32, each by itself and both."""
    rows_of_sizes(T, W, kind, [1e-3, 0.125, 1.0, 1e4, 1e15, 1e19, 1e30], size, eps)


@pytest.mark.parametrize("T,W", [(3, 96), (3, 2048), (200, 2048), (3, 8224)])
@pytest.mark.parametrize("x,d,eps", [(1.0, 1e36, 0.0), (1e18, 1e36, 1.0)])
def test_norm_backward_where_large_products_cancel(cuda_dev, T, W, x, d, eps):
    alternating(T, W, x, d, eps)


def alternating(T, W, x, d, eps):
    """Rows of one value with gradients of alternating signs: a sum of 0 of large or small terms."""
    s = np.full((T, W), x)
    dn = np.full((T, W), d) * np.where(np.arange(W) % 2, 1.0, -1.0)
    dn[1] = 0.0
    dn[2, 5] *= 3
    assert check_norm(*norm_backward(s, dn, np.ones(W), eps, "float32"), "float32", T, W).all()


@pytest.mark.parametrize("W", [96, 7168])
def test_norm_backward_of_one_value_far_above_its_row(cuda_dev, W):
    r = np.random.default_rng(6)
    x, dn = r.normal(size=(4, W)), np.abs(r.normal(size=(4, W))) * 1e35
    x[0, 3], dn[0, 3] = 1e21, 0.0
    x[1, 64], dn[1, 64] = 1e30, 0.0
    x[2, 40] = -1e25
    dn *= np.sign(x)
    for kind in sorted(TYPES):
        assert check_norm(*norm_backward(x, dn, np.ones(W), 1e-5, kind), kind, 4, W).all()


@pytest.mark.parametrize("T,W", NORM_SHAPES)
@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("size", [1e-30, 1e-10, 1.0, 1e20, 3e35])
@pytest.mark.parametrize("eps", [0.0, 1e-5])
def test_norm_backward_of_small_rows(cuda_dev, T, W, kind, size, eps):
    """Sums of squares and of products that are below fp32's normal numbers, each by itself and both."""
    rows_of_sizes(T, W, kind, [1e-36, 1e-30, 1e-23, 1e-18, 1e-13, 1e-10, 1e-5, 1.0, 1e30], size, eps)


@pytest.mark.parametrize("T,W", [(3, 96), (3, 2048), (200, 2048), (3, 8224)])
@pytest.mark.parametrize("x,d,eps", [(1e-15, 1e20, 0.0), (1e-15, 1e20, 1e-30), (1e-20, 0.0, 0.0), (1e-36, 0.0, 0.0), (1e-25, 1e10, 0.0),
                                     (1e-15, 1e-30, 0.0), (1e-30, 1e-37, 0.0)])
def test_norm_backward_where_products_of_small_rows_cancel(cuda_dev, T, W, x, d, eps):
    alternating(T, W, x, d, eps)


@pytest.mark.parametrize("T,W", [(3, 96), (3, 2048), (200, 2048), (3, 8224), (3, 16416)])
@pytest.mark.parametrize("kind", sorted(TYPES))
def test_norm_backward_of_small_rows_with_large_gradients_at_zeros(cuda_dev, T, W, kind):
    """Gradients that no scaled product may take part in, where s is 0, beside products of 1e-44."""
    r = np.random.default_rng(9)
    s, dn = np.abs(r.normal(size=(T, W))) * 1e-14, np.abs(r.normal(size=(T, W))) * 1e-30
    s[:, 5::32], dn[:, 5::32] = 0.0, 1e12
    assert check_norm(*norm_backward(s, dn, np.ones(W), 0.0, kind), kind, T, W).all() and k3mx.k3mx_device_status() == (0, 0)
