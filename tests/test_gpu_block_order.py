"""The order of a sum over a token's pairs does not depend on the other tokens of the call."""
import numpy as np
import pytest
import torch

import mxfp4_routed_expert_k3mx_gb300 as k3mx
from test_gpu_block_pairs import DEV, TYPES, placed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [1, 2, 3, 6, 8, 9, 16, 17, 33, 40])
@pytest.mark.parametrize("T,W", [(1100, 256), (40, 7168), (64, 1000), (5000, 64), (50, 8200)])
@pytest.mark.parametrize("rows_type", sorted(TYPES))
@pytest.mark.parametrize("y_type", sorted(TYPES))
def test_a_token_alone_and_among_others(cuda_dev, K, T, W, rows_type, y_type):
    """The same bits, and those of the products added with K rising, the base last."""
    place, R = placed(T, K, 0.2, K + W)
    gen = torch.Generator(device=DEV).manual_seed(K)
    normal = lambda *s: torch.randn(*s, generator=gen, device=DEV)
    rows, w, base = normal(R, W).to(TYPES[rows_type]), normal(T, K), normal(T, W).to(TYPES[y_type])
    at = torch.from_numpy(place).to(DEV)
    y = torch.empty_like(base)
    k3mx.k3mx_combine(y, rows, at, w=w, base=base)
    for t in (0, T // 2, T - 1):
        one = torch.empty_like(y[:1])
        k3mx.k3mx_combine(one, rows, at[t:t + 1], w=w[t:t + 1], base=base[t:t + 1])
        assert torch.equal(one, y[t:t + 1])
        # a fused product and sum rounds once: in doubles the product is exact, the sum nearly, and fp32's rounding of it
        # is the fused one's but where the double's own rounding led to a tie
        acc = torch.zeros(W, device=DEV)
        for k in range(K):
            if place[t, k] >= 0:
                acc = (w[t, k].double() * rows[place[t, k]].double() + acc.double()).float()
        want = (acc + base[t].float()).to(TYPES[y_type])
        assert (one[0] != want).sum() <= 1
    few = torch.empty_like(y[:7])
    k3mx.k3mx_combine(few, rows, at[:7], w=w[:7], base=base[:7])
    assert torch.equal(few, y[:7]) and k3mx.k3mx_device_status() == (0, 0)
