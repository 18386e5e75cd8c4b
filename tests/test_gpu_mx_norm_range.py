"""The norm over the whole range its header names: root mean squares from 2^-63
to 2^120, so that the squares' sum (and single squares) leave fp32 while the
result is ordinary.  Within the header's 2^-20 of double precision, by the checks
of the other norm tests."""
import pytest
import torch

from test_gpu_mx_format import BF16, F32, check_norm, run_norm

pytestmark = pytest.mark.gpu

# one form of the kernel each: a row to a warp (one and four runs a lane), to a CTA (one, two, four runs a thread)
SHAPES = [(5, 64), (700, 64), (40, 1024), (20, 7168), (1000, 7168), (9, 16384), (2, 32768)]


def rows(t, d, rms, dtype, seed):
    g = torch.Generator(device="cuda:0").manual_seed(seed)
    v = torch.randn(t, d, generator=g, device="cuda:0", dtype=torch.float64)
    return (v * rms).to(dtype), (1 + 0.2 * torch.randn(d, generator=g, device="cuda:0")).to(BF16)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,d", SHAPES)
@pytest.mark.parametrize("e", [-61, 52, 56, 59, 62, 64, 80, 118])
def test_root_mean_squares_of_any_size(cuda_dev, dtype, t, d, e):
    x, w = rows(t, d, 2.0 ** e, dtype, d + t)
    check_norm(x, None, w, 0.0)
    r, _ = rows(t, d, 2.0 ** e, dtype, d + t + 1)
    check_norm(x, r, w, 1e-5, normed=False) if e > 0 else check_norm(x, r, w, 0.0, normed=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,d", SHAPES)
def test_rows_on_either_side_of_the_overflow(cuda_dev, dtype, t, d):
    """Equal magnitudes whose squares add up to just below and just above 2^128,
    a single large value in an ordinary row, and ordinary rows between them."""
    x, w = rows(t, d, 1.0, dtype, t * d)
    edge = 2.0 ** 64 / d ** 0.5
    for i, f in enumerate((0.97, 0.999, 1.0, 1.001, 1.03)):
        if i < t:
            x[i] = torch.sign(x[i].float()).to(dtype) * f * edge
    if t > 6:
        x[5, d // 2], x[6, 0], x[t - 1, d - 1] = 2.0 ** 63.5, -2.0 ** 66, 2.0 ** 65
    check_norm(x, None, w, 1e-5)
    # ordinary rows beside them are what they are alone
    if 8 < t <= 64:                                        # (one row and t rows take the same form)
        alone = run_norm(x[7:8].contiguous(), None, w, 1e-5)
        among = run_norm(x, None, w, 1e-5)
        assert torch.equal(among[0][7:8], alone[0]) and torch.equal(among[1][7:8], alone[1])


def test_large_eps(cuda_dev):
    """eps beside which the mean square is little, up to where their sum leaves
    fp32."""
    x, w = rows(6, 512, 1.0, F32, 1)
    for eps in (1.0, 1e30, 3.3e38):
        check_norm(x, None, w, eps)
    x, w = rows(6, 512, 2.0 ** 59, F32, 2)
    check_norm(x, None, w, 3.4e38)
