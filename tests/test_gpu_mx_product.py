"""Dense and grouped products of MXFP8 activations with MXFP4 weights against
double precision: |error| <= 1e-5 * sum |x w| (the header's bound), plus
y's rounding (half a bf16 ulp: 2^-9 relative, doubled for the value it is
taken of)."""
import numpy as np
import pytest
import torch

import mx_ref
import mxfp4_routed_expert_k3mx_gb300 as k3mx

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def inputs(rows, inner, shape, seed, nan_frac=0.02):
    rng = np.random.default_rng(seed)
    xc = rng.integers(0, 256, (rows, inner)).astype(np.uint8)
    xc[(xc & 127) == 127] = 8
    xs = rng.integers(115, 130, (rows, inner // 32)).astype(np.uint8)
    p = rng.integers(0, 256, shape + (inner // 2,)).astype(np.uint8)
    ws = rng.integers(112, 132, shape + (inner // 32,)).astype(np.uint8)
    ws[rng.random(ws.shape) < nan_frac] = 255
    return xc, xs, p, ws


def dev(*arrays):
    return [torch.from_numpy(a).to("cuda:0") for a in arrays]


def assert_close(got, y, absdot, dtype, what=""):
    got = got.double().cpu().numpy()
    bound = 1e-5 * absdot + (2.0 ** -8 * np.abs(y) if dtype == BF16 else 0.0) + 2.0 ** -140
    err = np.abs(got - y)
    assert np.all(err <= bound), f"{what}: {np.sum(~(err <= bound))} of {err.size} off, worst {np.max(err / bound)}"


def linear(xc, xs, p, ws, dtype):
    y = torch.full((xc.shape[0], p.shape[0]), float("nan"), dtype=dtype, device="cuda:0")
    return k3mx.k3mx_mx_linear(y, *dev(xc, xs, p, ws))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,inner,out", [
    (1, 128, 1), (1, 128, 129), (1, 7168, 300), (3, 256, 64), (8, 640, 127), (9, 640, 128), (17, 1152, 130),
    (32, 2048, 1000), (33, 3584, 100), (64, 896, 2049), (128, 384, 256), (129, 1280, 257), (255, 512, 96),
    (257, 128, 384), (300, 1152, 1000), (1000, 512, 300), (2, 16384, 40), (520, 4096, 40)])
def test_linear(cuda_dev, dtype, rows, inner, out):
    a = inputs(rows, inner, (out,), rows + inner + out)
    got = linear(*a, dtype)
    y, ad = mx_ref.product(*a)
    assert_close(got, y, ad, dtype)
    assert k3mx.k3mx_device_status() == (0, 0)


def test_linear_is_exact_on_small_integers_and_deterministic(cuda_dev):
    """Integer codes under unit scales: every partial sum is an integer below
    2^24, so the product is exact in any order."""
    rng = np.random.default_rng(3)
    grid = np.array([0, 0x38, 0x40, 0x48, 0xB8, 0xC0], np.uint8)     # 0, 1, 2, 4, -1, -2 in e4m3
    for rows, inner, out in ((5, 1024, 200), (200, 512, 333), (700, 768, 256)):
        xc = grid[rng.integers(0, len(grid), (rows, inner))]
        code = np.array([0, 2, 4, 5, 6, 10, 12], np.uint8)[rng.integers(0, 7, (out, inner))]   # 0 1 2 3 4 -1 -2
        p, s1, s2 = mx_ref.pack(code), np.full((rows, inner // 32), 127, np.uint8), np.full((out, inner // 32), 127, np.uint8)
        y, _ = mx_ref.product(xc, s1, p, s2)
        got = linear(xc, s1, p, s2, F32)
        assert np.array_equal(got.cpu().numpy(), y.astype(np.float32))
    a = inputs(100, 3584, (500,), 9)
    assert torch.equal(linear(*a, F32), linear(*a, F32))


def test_linear_one_hot_rows_read_single_columns(cuda_dev):
    """Row t holds one 1 in column t * 37 % inner: y[t] is that column of w."""
    inner, out, rows = 1280, 137, 150
    rng = np.random.default_rng(4)
    col = np.arange(rows) * 37 % inner
    xc = np.zeros((rows, inner), np.uint8)
    xc[np.arange(rows), col] = 0x38
    xs = np.full((rows, inner // 32), 127, np.uint8)
    p = rng.integers(0, 256, (out, inner // 2)).astype(np.uint8)
    ws = rng.integers(100, 150, (out, inner // 32)).astype(np.uint8)
    w = mx_ref.values(mx_ref.unpack(p), ws, 0)
    assert np.array_equal(linear(xc, xs, p, ws, F32).cpu().numpy(), w[:, col].T.astype(np.float32))


@pytest.mark.parametrize("rows", [1, 40, 200, 400])
def test_linear_scale_edges(cuda_dev, rows):
    """Scale bytes at the ends of the range whose products stay in fp32, rows
    of nothing but dropped blocks, a NaN scale and a NaN code in x."""
    xc, xs, p, ws = inputs(rows, 512, (150,), 5, nan_frac=0.0)
    xs[:], ws[:] = 127, 127
    ws[3], ws[4, :8], ws[140] = 255, 255, 0
    ws[5], xs[0] = 1, 130
    ws[6] = 230                     # 2^103: sums stay below 2^103 * 512 * 6 * 448 * 8 < 2^127
    y, ad = mx_ref.product(xc, xs, p, ws)
    got = linear(xc, xs, p, ws, F32)
    assert torch.all(got[:, 3] == 0)
    assert_close(got, y, ad, F32)
    ws[6] = 127
    xs[rows - 1, 7] = 255
    xc[rows // 2, 300] = 0x7F
    got = linear(xc, xs, p, ws, F32)
    bad = sorted({rows - 1, rows // 2})
    assert torch.isnan(got[bad]).all()
    keep = [r for r in range(rows) if r not in bad]
    if keep:
        y, ad = mx_ref.product(xc[keep], xs[keep], p, ws)
        assert_close(got[keep], y, ad, F32)


# --------------------------------------------------------------- grouped --

def grouped_reference(a, offsets, out, fill):
    xc, xs, p, ws = a
    y = np.full((xc.shape[0], out), fill)
    ad = np.zeros_like(y)
    for g in range(len(offsets) - 1):
        lo, hi = offsets[g], offsets[g + 1]
        if hi > lo:
            y[lo:hi], ad[lo:hi] = mx_ref.product(xc[lo:hi], xs[lo:hi], p[g], ws[g])
    return y, ad


def check_grouped(counts, inner, out, dtype, before=0, after=0, seed=0):
    offsets = np.concatenate([[before], before + np.cumsum(counts)]).astype(np.int32)
    rows = int(offsets[-1]) + after
    a = inputs(rows, inner, (len(counts), out), seed + rows)
    y = torch.full((rows, out), -7.0, dtype=dtype, device="cuda:0")
    k3mx.k3mx_mx_grouped(y, *dev(*a, offsets))
    ref, ad = grouped_reference(a, offsets, out, -7.0)
    assert_close(y, ref, ad, dtype, f"{counts}")
    inside = slice(before, rows - after)
    assert torch.all(y[:before] == -7.0) and torch.all(y[rows - after:] == -7.0) and not torch.all(y[inside] == -7.0)
    assert k3mx.k3mx_device_status() == (0, 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("counts,inner,out", [
    ([1], 128, 1), ([0, 1, 0], 256, 130), ([5, 0, 0, 3, 1], 640, 128), ([1] * 16, 3584, 200),
    ([8, 9, 7, 16, 17, 33], 512, 129), ([0, 300, 0, 1, 130, 0], 1152, 257), ([256, 257, 255, 31], 384, 96),
    ([0] * 63 + [40], 128, 64), ([3, 600, 2], 896, 500)])
def test_grouped(cuda_dev, dtype, counts, inner, out):
    check_grouped(counts, inner, out, dtype)


def test_grouped_leaves_rows_of_no_group(cuda_dev):
    check_grouped([4, 0, 60, 9], 256, 140, F32, before=5, after=11)
    check_grouped([1, 2], 1024, 33, BF16, before=300, after=1)


def test_grouped_many_groups_and_all_empty(cuda_dev):
    rng = np.random.default_rng(1)
    check_grouped(list(rng.integers(0, 4, 1024)), 128, 48, F32)
    xc, xs, p, ws = inputs(6, 128, (3, 40), 2)
    y = torch.full((6, 40), -7.0, device="cuda:0")
    k3mx.k3mx_mx_grouped(y, *dev(xc, xs, p, ws, np.full(4, 6, np.int32)))
    assert torch.all(y == -7.0)


def test_grouped_equals_linear(cuda_dev):
    """One group of all rows gives the dense product."""
    for rows, inner, out in ((3, 512, 300), (70, 1024, 200), (600, 640, 130)):
        a = inputs(rows, inner, (out,), rows)
        y = torch.empty(rows, out, device="cuda:0")
        k3mx.k3mx_mx_grouped(y, *dev(a[0], a[1], a[2][None], a[3][None], np.array([0, rows], np.int32)))
        ref, ad = mx_ref.product(*a)
        assert_close(y, ref, ad, F32)


@pytest.mark.parametrize("offsets,bad,good", [
    ([0, 5, 3, 9], 1, [0, 2]), ([0, 4, 8, 40], 2, [0, 1]), ([-2, 4, 8, 9], 0, [1, 2])])
def test_grouped_refuses_offsets_on_the_device(cuda_dev, offsets, bad, good):
    """A group whose offsets fall or leave the rows is skipped and reported;
    nothing outside the arrays is touched and the other groups are done."""
    k3mx.k3mx_device_status()
    a = inputs(9, 256, (3, 70), 8)
    y = torch.full((9, 70), -7.0, device="cuda:0")
    k3mx.k3mx_mx_grouped(y, *dev(*a, np.array(offsets, np.int32)))
    assert k3mx.k3mx_device_status() == (1, bad)
    for g in good:
        # (of offsets that fall, rows claimed by two groups hold one of the two products)
        lo = max([offsets[g]] + [offsets[h + 1] for h in good if h < g])
        hi = min([offsets[g + 1]] + [offsets[h] for h in good if h > g])
        ref, ad = mx_ref.product(a[0][lo:hi], a[1][lo:hi], a[2][g], a[3][g])
        assert_close(y[lo:hi], ref, ad, F32)


def test_products_on_another_stream(cuda_dev):
    a = inputs(50, 1024, (300,), 11)
    s = torch.cuda.Stream()
    d = dev(*a)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        y = torch.empty(50, 300, device="cuda:0")
        k3mx.k3mx_mx_linear(y, *d)
    y2 = torch.empty(50, 300, device="cuda:0")
    k3mx.k3mx_mx_linear(y2, *d, stream=s)
    s.synchronize()
    ref, ad = mx_ref.product(*a)
    assert_close(y, ref, ad, F32)
    assert torch.equal(y, y2)


def test_norm_quantize_product_chain(cuda_dev):
    """rmsnorm -> product with weights that the quantiser made, against the
    chain of definitions on the codes that the GPU wrote."""
    t, d, n = 19, 1152, 260
    x, r = torch.randn(t, d, device="cuda:0").to(BF16), torch.randn(t, d, device="cuda:0").to(BF16)
    w = torch.randn(n, d, device="cuda:0")
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda:0")
    p, ws, c, s = u8(n, d // 2), u8(n, d // 32), u8(t, d), u8(t, d // 32)
    y = torch.empty(t, n, device="cuda:0")
    k3mx.k3mx_mx_quantize(p, ws, w, k3mx.K3MX_MXFP4)
    k3mx.k3mx_rmsnorm_mx(c, s, torch.empty_like(x), x, r, torch.ones(d, dtype=BF16, device="cuda:0"), 1e-5)
    k3mx.k3mx_mx_linear(y, c, s, p, ws)
    ref, ad = mx_ref.product(*[v.cpu().numpy() for v in (c, s, p, ws)])
    assert_close(y, ref, ad, F32)


def test_products_in_a_graph(cuda_dev):
    """Captured once, replayed on changed inputs."""
    a = inputs(40, 1024, (300,), 21)
    d = dev(*a)
    y = torch.empty(40, 300, device="cuda:0")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        k3mx.k3mx_mx_linear(y, *d)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            k3mx.k3mx_mx_linear(y, *d)
        b = inputs(40, 1024, (300,), 22)
        for t, n in zip(d, dev(*b)):
            t.copy_(n)
        g.replay()
        s.synchronize()
    ref, ad = mx_ref.product(*b)
    assert_close(y, ref, ad, F32)


def test_product_reads_what_the_kernel_before_wrote(cuda_dev):
    """Weights, activations and offsets written by the launches right before
    the product on the stream, many times over with changing values."""
    rng = np.random.default_rng(5)
    t, inner, out = 3, 512, 256
    w = [torch.from_numpy(rng.standard_normal((out, inner)).astype(np.float32)).to("cuda:0") for _ in range(2)]
    x = [torch.from_numpy(rng.standard_normal((t, inner)).astype(np.float32)).to("cuda:0") for _ in range(2)]
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda:0")
    ref = []
    for i in range(2):
        p, ws, c, s = u8(out, inner // 2), u8(out, inner // 32), u8(t, inner), u8(t, inner // 32)
        k3mx.k3mx_mx_quantize(p, ws, w[i], k3mx.K3MX_MXFP4)
        k3mx.k3mx_mx_quantize(c, s, x[i], k3mx.K3MX_MXFP8)
        torch.cuda.synchronize()
        y = torch.empty(t, out, device="cuda:0")
        k3mx.k3mx_mx_linear(y, c, s, p, ws)
        torch.cuda.synchronize()
        ref.append(y)
    ys = [torch.empty(t, out, device="cuda:0") for _ in range(200)]
    for i, y in enumerate(ys):
        k3mx.k3mx_mx_quantize(c, s, x[i % 2], k3mx.K3MX_MXFP8)
        k3mx.k3mx_mx_quantize(p, ws, w[i % 2], k3mx.K3MX_MXFP4)
        k3mx.k3mx_mx_linear(y, c, s, p, ws)
    torch.cuda.synchronize()
    assert all(torch.equal(y, ref[i % 2]) for i, y in enumerate(ys))


@pytest.mark.parametrize("rows,inner,out", [(2, 65536, 1000), (40, 65536, 1000), (100, 65536, 300), (300, 65536, 300)])
def test_product_waits_are_bounded(cuda_dev, rows, inner, out):
    """With a limit of one poll a wait gives up (the epilogue's, for bf16 sums
    of 512 tiles in one accumulation, lasts many polls): the status says so,
    nothing faults, and with the limit restored the next call is right."""
    a = inputs(rows, inner, (out,), rows)
    d = dev(*a)
    clean = torch.empty(rows, out, dtype=BF16, device="cuda:0")
    k3mx.k3mx_mx_linear(clean, *d)
    assert k3mx.k3mx_device_status() == (0, 0)
    y = torch.empty_like(clean)
    k3mx.k3mx_set_wait_limit(1)
    try:
        seen = 0
        for _ in range(50):
            k3mx.k3mx_mx_linear(y, *d)
            st, detail = k3mx.k3mx_device_status()
            assert st in (0, 6), (st, detail)
            if st == 6:
                assert 400 <= detail < 460
                seen += 1
                break
    finally:
        k3mx.k3mx_set_wait_limit(0)
    assert seen, "no wait ran out"
    y.fill_(0)
    k3mx.k3mx_mx_linear(y, *d)
    assert k3mx.k3mx_device_status() == (0, 0)
    assert torch.equal(y, clean)


@pytest.mark.parametrize("rows", [2, 40, 300])
def test_waits_for_dropped_blocks_are_bounded(cuda_dev, rows):
    """The same where every fourth block is dropped, so that the scales' warp
    also waits for tiles: whichever wait gives up, the call ends, and the next
    one with the limit restored is right."""
    xc, xs, p, ws = inputs(rows, 65536, (300,), rows)
    ws[:, ::4] = 255
    d = dev(xc, xs, p, ws)
    clean = torch.empty(rows, 300, dtype=BF16, device="cuda:0")
    k3mx.k3mx_mx_linear(clean, *d)
    assert k3mx.k3mx_device_status() == (0, 0)
    y = torch.empty_like(clean)
    k3mx.k3mx_set_wait_limit(1)
    try:
        seen = set()
        for _ in range(20):
            k3mx.k3mx_mx_linear(y, *d)
            seen.add(k3mx.k3mx_device_status())
    finally:
        k3mx.k3mx_set_wait_limit(0)
    assert all(st == 0 or st == 6 and 400 <= detail < 460 for st, detail in seen), seen
    assert any(st == 6 for st, _ in seen), "no wait ran out"
    y.fill_(0)
    k3mx.k3mx_mx_linear(y, *d)
    assert k3mx.k3mx_device_status() == (0, 0)
    assert torch.equal(y, clean)


# ------------------------------------------------- offsets past 32 bits --

def test_grouped_weights_past_4_gib(cuda_dev):
    """Group 70 of 72 matrices of 64 MiB: its codes start past 2^32 bytes."""
    E, out, inner, rows = 72, 8192, 16384, 5
    packed = torch.zeros(E, out, inner // 2, dtype=torch.uint8, device="cuda:0")
    wscales = torch.full((E, out, inner // 32), 120, dtype=torch.uint8, device="cuda:0")
    gen = torch.Generator(device="cuda:0").manual_seed(0)
    packed[70] = torch.randint(0, 256, (out, inner // 2), generator=gen, device="cuda:0", dtype=torch.uint8)
    packed[69] = 0x11
    xc, xs, _, _ = inputs(rows, inner, (1,), 3)
    off = np.array([0] * 70 + [2, rows, rows], np.int32)          # group 69: rows 0-1, group 70: rows 2-4
    y = torch.empty(rows, out, device="cuda:0")
    k3mx.k3mx_mx_grouped(y, *dev(xc, xs), packed, wscales, torch.from_numpy(off).to("cuda:0"))
    pick = np.array([0, 1, 127, 128, 5000, 8190, 8191])
    for g, lo, hi in ((69, 0, 2), (70, 2, rows)):
        ref, ad = mx_ref.product(xc[lo:hi], xs[lo:hi], packed[g, pick].cpu().numpy(), wscales[g, pick].cpu().numpy())
        assert_close(y[lo:hi][:, pick], ref, ad, F32)


def test_linear_output_past_4_gib(cuda_dev):
    """y of 2^31 + elements: the last rows lie past 2^32 bytes."""
    rows, inner, out = 70_000, 128, 32_768
    xc, xs, p, ws = inputs(rows, inner, (out,), 9)
    y = torch.empty(rows, out, dtype=BF16, device="cuda:0")
    k3mx.k3mx_mx_linear(y, *dev(xc, xs, p, ws))
    pick = np.array([0, 1, 255, 256, 40_000, 65_535, 65_536, 69_998, 69_999])
    ref, ad = mx_ref.product(xc[pick], xs[pick], p, ws)
    assert_close(y[torch.from_numpy(pick).to("cuda:0")], ref, ad, BF16)
