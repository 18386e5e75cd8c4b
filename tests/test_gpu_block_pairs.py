"""Pairs by expert, rows there and back, and their gradients, against the
double-precision definitions."""
import numpy as np
import pytest
import torch

import block_ref
import mxfp4_routed_expert_k3mx_gb300 as k3mx

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16}


def i32(*shape, fill=-7):
    return torch.full(shape, fill, dtype=torch.int32, device=DEV)


def doubles(t):
    return t.detach().cpu().double().numpy()


def workspace(n):
    return torch.empty(n, dtype=torch.uint8, device=DEV) if n else None


def sorted_pairs(idx, n):
    T, K = idx.shape
    offsets, perm, place = i32(n + 1), i32(T * K), i32(T, K)
    k3mx.k3mx_sort(offsets, perm, place, idx, workspace(k3mx.k3mx_sort_workspace_size(T, K, n)))
    return offsets, perm, place


def choices(T, K, n, drop, seed, skew=1.0):
    """Experts with repetitions, few of them popular, some dropped."""
    r = np.random.default_rng(seed)
    p = np.exp(skew * r.normal(size=n))
    idx = r.choice(n, size=(T, K), p=p / p.sum())
    return np.where(r.random((T, K)) < drop, -1, idx).astype(np.int32)


# ------------------------------------------------------------------- sort --

@pytest.mark.parametrize("T,K,n,drop", [
    (1, 1, 1, 0.0), (1, 16, 896, 0.0), (1, 16, 896, 1.0), (2, 3, 4, 0.3), (31, 1, 1024, 0.0), (33, 1, 5, 0.5), (64, 16, 896, 0.1),
    (1000, 7, 24, 0.2), (512, 16, 896, 0.0), (8192, 1, 3, 0.0), (8193, 1, 1, 0.0), (683, 12, 100, 0.9), (4096, 16, 896, 0.1),
    (16385, 16, 1024, 0.0), (70001, 4, 37, 0.3), (300000, 1, 1024, 0.0), (1, 20000, 33, 0.1), (65536, 16, 896, 0.05), (256, 1, 9, 0.1), (257, 1, 9, 0.1), (2048, 1, 50, 0.0), (2049, 1, 50, 0.1),
    (4096, 1, 50, 0.0), (4097, 1, 50, 0.1), (16384, 1, 7, 0.0), (16385, 1, 7, 0.1), (65537, 1, 33, 0.0), (131073, 1, 33, 0.1)])
def test_sort(cuda_dev, T, K, n, drop):
    idx = choices(T, K, n, drop, seed=T + K)
    offsets, perm, place = sorted_pairs(torch.from_numpy(idx).to(DEV), n)
    assert k3mx.k3mx_device_status() == (0, 0)
    flat = idx.reshape(-1)
    order = np.argsort(np.where(flat < 0, n, flat), kind="stable")
    live = int((flat >= 0).sum())
    if T * K < 1000:
        want = block_ref.sort(idx, n)
        assert np.array_equal(want[1], order[:live])
        assert np.array_equal(place.cpu().numpy(), want[2]) and np.array_equal(offsets.cpu().numpy(), want[0])
    assert np.array_equal(offsets.cpu().numpy(), np.searchsorted(np.sort(flat[flat >= 0]), np.arange(n + 1)))
    perm = perm.cpu().numpy()
    assert np.array_equal(perm[:live], order[:live]) and np.all(perm[live:] == -7)       # behind the last: left
    want = np.full(T * K, -1)
    want[order[:live]] = np.arange(live)
    assert np.array_equal(place.cpu().numpy().reshape(-1), want)


@pytest.mark.parametrize("T,K", [(1 << 24, 1), (1 << 20, 16)])
def test_sort_of_the_most_pairs(cuda_dev, T, K):
    gen = torch.Generator(device=DEV).manual_seed(3)
    idx = torch.randint(-1, 1024, (T, K), generator=gen, device=DEV, dtype=torch.int32)
    offsets, perm, place = sorted_pairs(idx, 1024)
    key, order = torch.sort(torch.where(idx < 0, torch.full_like(idx, 1024), idx).reshape(-1), stable=True)
    n = int(offsets[-1])
    assert torch.equal(offsets.long(), torch.searchsorted(key, torch.arange(1025, device=DEV, dtype=torch.int32)))
    assert torch.equal(perm[:n].long(), order[:n]) and torch.all(perm[n:] == -7)
    want = torch.full((T * K,), -1, dtype=torch.int32, device=DEV)
    want[order[:n]] = torch.arange(n, dtype=torch.int32, device=DEV)
    assert torch.equal(place.reshape(-1), want) and k3mx.k3mx_device_status() == (0, 0)


def test_sort_without_perm_and_with_a_larger_workspace(cuda_dev):
    idx = torch.from_numpy(choices(30000, 5, 60, 0.1, 1)).to(DEV)
    want = sorted_pairs(idx, 60)
    offsets, place = i32(61), i32(30000, 5)
    k3mx.k3mx_sort(offsets, None, place, idx, torch.empty(1 << 16, dtype=torch.int64, device=DEV))
    assert torch.equal(offsets, want[0]) and torch.equal(place, want[2])
    few = torch.zeros(3, 2, dtype=torch.int32, device=DEV)
    k3mx.k3mx_sort(i32(61), None, i32(3, 2), few, None)
    with pytest.raises(k3mx.K3mxError, match="EWORKSPACE"):
        k3mx.k3mx_sort(i32(61), None, i32(30000, 5), idx, None)


@pytest.mark.parametrize("T", [5, 5000, 30000, 100000])
def test_sort_reports_a_bad_expert_and_drops_its_pair(cuda_dev, T):
    idx = choices(T, 2, 9, 0.0, 3)
    good = idx.copy()
    idx[3, 1], good[3, 1] = 9, -1
    offsets, perm, place = sorted_pairs(torch.from_numpy(idx).to(DEV), 9)
    assert k3mx.k3mx_device_status() == (1, 7)
    want = sorted_pairs(torch.from_numpy(good).to(DEV), 9)
    assert all(torch.equal(a, b) for a, b in zip((offsets, perm, place), want))
    idx[3, 1] = -2
    sorted_pairs(torch.from_numpy(idx).to(DEV), 9)
    assert k3mx.k3mx_device_status() == (1, 7)


def test_sort_agrees_with_group(cuda_dev):
    idx = torch.from_numpy(choices(777, 16, 896, 0.1, 5)).to(DEV)
    offsets, perm, place = sorted_pairs(idx, 896)
    o2, p2 = i32(897), i32(777 * 16)
    k3mx.k3mx_group(i32(896), o2, p2, idx, workspace(k3mx.k3mx_group_workspace_size(777)))
    n = int(offsets[-1])
    assert torch.equal(offsets, o2) and torch.equal(perm[:n], p2[:n])


# ---------------------------------------------------------- there and back --

def placed(T, K, drop, seed, extra=3):
    """place of T x K pairs in rows of which `extra` and the dropped ones' are named by none."""
    r = np.random.default_rng(seed)
    R = T * K + extra
    place = r.permutation(R)[:T * K].reshape(T, K).astype(np.int32)
    return np.where(r.random((T, K)) < drop, -1, place).astype(np.int32), R


SHAPES = [(1, 1, 1), (1, 16, 3584), (1, 2, 7168), (3, 5, 1), (7, 3, 33), (5, 4, 64), (64, 2, 8), (300, 6, 1000), (257, 1, 1001),
          (33, 17, 520), (2, 64, 4100), (1024, 8, 256), (70, 40, 4096), (5000, 33, 64), (9, 40, 33), (300, 5, 1001), (700, 2, 9), (1000, 1, 5)]


@pytest.mark.parametrize("T,K,W", SHAPES)
@pytest.mark.parametrize("kind", ["float32", "bfloat16", "mxfp8"])
def test_dispatch(cuda_dev, T, K, W, kind):
    if kind == "mxfp8":
        W = (W + 31) // 32 * 32
    place, R = placed(T, K, 0.2, T + W)
    gen = torch.Generator(device=DEV).manual_seed(W)
    for pad in (0, 16, 5):
        wide = torch.randint(0, 256, (T, (W + pad) * 4), generator=gen, device=DEV, dtype=torch.uint8)
        x = (wide[:, :W + pad] if kind == "mxfp8" else wide.view(torch.int32).float().to(TYPES[kind])[:, :W + pad]).contiguous()[:, :W]
        rows = torch.full((R, W), 99, dtype=x.dtype, device=DEV)
        xs = torch.randint(0, 256, (T, W // 32), generator=gen, device=DEV, dtype=torch.uint8) if kind == "mxfp8" else None
        scales = torch.full((R, W // 32), 98, dtype=torch.uint8, device=DEV) if kind == "mxfp8" else None
        k3mx.k3mx_dispatch(rows, x, torch.from_numpy(place).to(DEV), scales=scales, x_scales=xs)
        want, ws = torch.full_like(rows, 99).cpu(), None if xs is None else torch.full_like(scales, 98).cpu()
        t, k = np.nonzero(place >= 0)
        want[place[t, k]] = x.cpu()[t]
        assert torch.equal(rows.cpu(), want)
        if xs is not None:
            ws[place[t, k]] = xs.cpu()[t]
            assert torch.equal(scales.cpu(), ws)
    assert k3mx.k3mx_device_status() == (0, 0)


@pytest.mark.parametrize("T,K,W", SHAPES)
@pytest.mark.parametrize("rows_type", sorted(TYPES))
@pytest.mark.parametrize("y_type", sorted(TYPES))
def test_combine_and_its_gradient(cuda_dev, T, K, W, rows_type, y_type):
    place, R = placed(T, K, 0.2, T + W)
    r = np.random.default_rng(T * K + W)
    at = torch.from_numpy(place).to(DEV)
    rows = torch.from_numpy(r.normal(size=(R, W))).to(TYPES[rows_type]).to(DEV)
    named = np.unique(place[place >= 0])
    rows[torch.from_numpy(np.setdiff1d(np.arange(R), named)).to(DEV)] = float("nan")      # nobody's rows are not read
    clean = np.nan_to_num(doubles(rows))
    w = torch.from_numpy(r.random((T, K)).astype(np.float32)).to(DEV)
    base = torch.from_numpy(r.normal(size=(T, W))).to(TYPES[y_type]).to(DEV)
    for ww, bb in ((w, None), (None, base), (w, base)):
        y = torch.full((T, W), float("nan"), dtype=TYPES[y_type], device=DEV)
        k3mx.k3mx_combine(y, rows, at, w=ww, base=bb)
        want, mag = block_ref.combine(clean, place, None if ww is None else doubles(ww), None if bb is None else doubles(bb))
        # K products and sums in fp32, each off by half a step of at most mag, and y's rounding of a value off by as much
        tol = (2 * K + 2) * 2.0 ** -24 * mag
        tol += block_ref.HALF[y_type] * (np.abs(want) + tol) + 1e-40
        assert np.all(np.abs(doubles(y) - want) <= tol)
    again = base.clone()
    k3mx.k3mx_combine(again, rows, at, w=w, base=again)                                   # in place
    assert torch.equal(again, y)
    for pad in (0, 8, 3):
        wide = torch.from_numpy(r.normal(size=(T, W + pad)) * 1e-3).to(TYPES[y_type]).to(DEV)
        dy = wide[:, :W]
        drows, dw = torch.full_like(rows, 77.0), torch.full_like(w, float("nan"))
        k3mx.k3mx_combine_backward(drows, dw, dy, rows, at, w)
        dr, want, mag = block_ref.combine_backward(doubles(dy), clean, place, doubles(w))
        # a lane adds at most W / 32 products in turn, lanes and warps in 13 more
        assert np.all(np.abs(doubles(dw) - want) <= (W / 32 + 16) * 2.0 ** -24 * mag + 1e-40)
        got, live = doubles(drows), place >= 0
        tol = (block_ref.HALF[rows_type] * (1 + 2.0 ** -20) + 2.0 ** -24) * np.abs(dr) + 1e-40
        assert np.all(np.abs(got[place[live]] - dr[live]) <= tol[live])
        assert np.all(got[np.setdiff1d(np.arange(R), named)] == 77.0)
        same, dw2 = rows.clone(), torch.empty_like(dw)
        k3mx.k3mx_combine_backward(same, dw2, dy, same, at, w)                            # in place
        assert torch.equal(dw2, dw) and torch.equal(same[at[at >= 0].long()], drows[at[at >= 0].long()])
    assert k3mx.k3mx_device_status() == (0, 0)


def test_combine_without_weights_is_dispatchs_gradient(cuda_dev):
    """<dispatch(x), g> = <x, combine(g)>, exactly for small whole numbers."""
    place, R = placed(50, 4, 0.3, 1, extra=0)
    at = torch.from_numpy(place).to(DEV)
    gen = torch.Generator(device=DEV).manual_seed(0)
    x, g = (torch.randint(-8, 9, (n, 96), generator=gen, device=DEV).float() for n in (50, R))
    rows, dx = torch.zeros(R, 96, device=DEV), torch.empty(50, 96, device=DEV)
    k3mx.k3mx_dispatch(rows, x, at)
    k3mx.k3mx_combine(dx, g, at)
    assert (rows * g).sum() == (x * dx).sum()


@pytest.mark.parametrize("W", [64, 33])
def test_a_token_without_pairs(cuda_dev, W):
    place = torch.full((3, 4), -1, dtype=torch.int32, device=DEV)
    rows, y = torch.full((2, W), float("inf"), device=DEV), torch.full((3, W), float("nan"), device=DEV)
    w = torch.full((3, 4), float("nan"), device=DEV)
    k3mx.k3mx_combine(y, rows, place, w=w)
    assert torch.all(y == 0)
    dw, drows = torch.full_like(w, 5.0), torch.full_like(rows, 4.0)
    k3mx.k3mx_combine_backward(drows, dw, torch.full_like(y, float("inf")), rows, place, w)
    assert torch.all(dw == 0) and torch.all(drows == 4.0)
    out = torch.full_like(rows, 3.0)
    k3mx.k3mx_dispatch(out, y, place)
    assert torch.all(out == 3.0) and k3mx.k3mx_device_status() == (0, 0)


def test_infinite_rows_and_weights_of_zero(cuda_dev):
    rows = torch.tensor([[float("inf")] * 8, [1.0] * 8, [float("nan")] * 8], device=DEV)
    place = torch.tensor([[0, 1], [2, 1], [1, -1]], dtype=torch.int32, device=DEV)
    y = torch.empty(3, 8, device=DEV)
    k3mx.k3mx_combine(y, rows, place, w=torch.tensor([[2.0, 1.0], [0.0, 1.0], [0.5, float("nan")]], device=DEV))
    assert torch.all(y[0] == float("inf")) and torch.all(y[1].isnan()) and torch.all(y[2] == 0.5)


@pytest.mark.parametrize("bad", [6, -2, 1 << 30, -(1 << 31)])
@pytest.mark.parametrize("W", [64, 30])
def test_a_place_outside_the_rows_is_reported_and_skipped(cuda_dev, bad, W):
    place = torch.tensor([[0, 1], [2, bad], [4, 5]], dtype=torch.int32, device=DEV)
    good = place.clone()
    good[1, 1] = -1
    x, w = torch.randn(3, W, device=DEV), torch.rand(3, 2, device=DEV)
    res = []
    for at in (place, good):
        rows, y, dr, dw = torch.zeros(6, W, device=DEV), torch.empty(3, W, device=DEV), torch.zeros(6, W, device=DEV), torch.empty(3, 2, device=DEV)
        want = (1, 3) if at is place else (0, 0)
        k3mx.k3mx_dispatch(rows, x, at)
        assert k3mx.k3mx_device_status() == want
        k3mx.k3mx_combine(y, rows, at, w=w)
        assert k3mx.k3mx_device_status() == want
        k3mx.k3mx_combine_backward(dr, dw, x, rows, at, w)
        assert k3mx.k3mx_device_status() == want
        res.append((rows, y, dr, dw))
    assert all(torch.equal(a, b) for a, b in zip(*res))


@pytest.mark.parametrize("off", [1, 4])
def test_rows_that_begin_off_sixteen_bytes(cuda_dev, off):
    place = torch.tensor([[0, 2], [1, -1]], dtype=torch.int32, device=DEV)
    flat = torch.randn(3 * 64 + off, device=DEV).bfloat16()
    rows, x, w = flat[off:].view(3, 64), torch.randn(2, 64, device=DEV).bfloat16(), torch.rand(2, 2, device=DEV)
    y, z = torch.empty(2, 64, device=DEV), torch.empty(2, 64, device=DEV)
    k3mx.k3mx_combine(y, rows, place, w=w)
    k3mx.k3mx_combine(z, rows.clone(), place, w=w)
    assert torch.equal(y, z)
    dr, ds, dw, dv = torch.zeros_like(flat)[off:].view(3, 64), torch.zeros(3, 64, device=DEV).bfloat16(), torch.empty_like(w), torch.empty_like(w)
    k3mx.k3mx_combine_backward(dr, dw, x, rows, place, w)
    k3mx.k3mx_combine_backward(ds, dv, x, rows.clone(), place, w)
    assert torch.equal(dr, ds) and torch.allclose(dw, dv, rtol=1e-5, atol=1e-5)
    k3mx.k3mx_dispatch(rows, x, place)
    assert torch.equal(rows[0], x[0]) and torch.equal(rows[2], x[0]) and torch.equal(rows[1], x[1])


@pytest.mark.parametrize("off,xoff", [(1, 0), (0, 3), (7, 9), (16, 4)])
def test_codes_that_begin_off_sixteen_bytes(cuda_dev, off, xoff):
    place, R = placed(9, 40, 0.3, off)                     # (more pairs a token than are listed at a time)
    gen = torch.Generator(device=DEV).manual_seed(off)
    u8 = lambda n: torch.randint(0, 256, (n,), generator=gen, device=DEV, dtype=torch.uint8)
    x, xs = u8(9 * 4224 + xoff)[xoff:].view(9, 4224), u8(9 * 132 + xoff)[xoff:].view(9, 132)
    rows, scales = u8(R * 4224 + off)[off:].view(R, 4224), u8(R * 132 + off)[off:].view(R, 132)
    want, ws = rows.cpu().clone(), scales.cpu().clone()
    k3mx.k3mx_dispatch(rows, x, torch.from_numpy(place).to(DEV), scales=scales, x_scales=xs)
    t, k = np.nonzero(place >= 0)
    want[place[t, k]], ws[place[t, k]] = x.cpu()[t], xs.cpu()[t]
    assert torch.equal(rows.cpu(), want) and torch.equal(scales.cpu(), ws)


def test_offsets_past_32_bits(cuda_dev):
    R, W = 700_000, 7168                                  # 5.0e9 elements
    rows = torch.empty(R, W, dtype=torch.bfloat16, device=DEV)
    place = torch.tensor([[R - 1, 3], [-1, R - 2]], dtype=torch.int32, device=DEV)
    x, w = torch.randn(2, W, device=DEV).bfloat16(), torch.tensor([[0.5, 0.25], [7.0, 2.0]], device=DEV)
    k3mx.k3mx_dispatch(rows, x, place)
    assert torch.equal(rows[R - 1], x[0]) and torch.equal(rows[3], x[0]) and torch.equal(rows[R - 2], x[1])
    y = torch.empty(2, W, device=DEV)
    k3mx.k3mx_combine(y, rows, place, w=w)
    assert torch.equal(y, torch.stack([0.75 * x[0].float(), 2.0 * x[1].float()]))
    dw = torch.empty_like(w)
    k3mx.k3mx_combine_backward(rows, dw, y.bfloat16(), rows, place, w)
    assert torch.equal(rows[R - 1], (0.5 * y[0].bfloat16().float()).bfloat16())
    assert torch.equal(rows[R - 2], (2.0 * y[1].bfloat16().float()).bfloat16())
    assert dw[1, 0] == 0 and torch.allclose(dw[1, 1], (y[1].bfloat16().double() * x[1].double()).sum().float(), rtol=1e-5)
    wide = torch.empty((1 << 32) + 64, dtype=torch.uint8, device=DEV)
    z = wide.as_strided((2, 64), (1 << 32, 1))            # a pitch of 2^32
    z.copy_(torch.arange(128, device=DEV, dtype=torch.uint8).view(2, 64))
    out, s = torch.zeros(2, 64, dtype=torch.uint8, device=DEV), torch.zeros(2, 2, dtype=torch.uint8, device=DEV)
    k3mx.k3mx_dispatch(out, z, torch.tensor([[0], [1]], dtype=torch.int32, device=DEV), scales=s, x_scales=s + 3)
    assert torch.equal(out, z) and torch.all(s == 3) and k3mx.k3mx_device_status() == (0, 0)
