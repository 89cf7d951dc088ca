"""Draws at temperatures and logits whose differences, or their ratio to the temperature, FP32 does not hold.

Against 64 bits with the tolerances of test_gpu_sample.check: differences here, scaled by a power of two or not, are exact to
2^-24 and carried on, so nothing is added to them."""
import math

import pytest
import torch
from test_gpu_sample import check
from test_gpu_verify_round import DEV, randn, vg  # noqa: F401

pytestmark = pytest.mark.gpu

WIDE = [torch.bfloat16, torch.float32]                   # whose range is FP32's


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("vocab", [9, 3001, 40007])
@pytest.mark.parametrize("T", [2.0 ** 63, 2.0 ** 64, 1e30, 1e37, 1e38, 3e38, math.inf])
def test_differences_past_the_range(vg, dtype, vocab, T):
    """The largest and the lowest value of the type in one row, and everything between."""
    g = torch.Generator().manual_seed(vocab)
    top, low = torch.finfo(dtype).max, torch.finfo(dtype).min
    x = torch.stack([randn(g, vocab).double() * s for s in (1e38, 1.0, 1e20, 3e38)]).clamp(low, top)
    x[:, 3], x[:, 5] = top, low
    x[1, ::2] = low
    x[2, ::2] = top
    x[3, 1::4] = -math.inf
    x = x.to(dtype)
    x[:, 3] = top
    u = torch.cat((torch.rand((4, 5), generator=g), torch.tensor([[0.0, 0.999, 1 - 2.0 ** -24]]).expand(4, 3)), 1).to(DEV)
    check(vg, x, u, T=[T] * 4)
    check(vg, x, u, T=[T] * 4, k=[vocab // 2] * 4, p=[0.7] * 4)
    check(vg, x, u, T=[T] * 4, k=[5] * 4, p=[0.9] * 4, mp=[0.01] * 4)


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("vocab", [9, 3001, 40007])
@pytest.mark.parametrize("T,scale", [(2.0 ** -119, 2.0 ** -118), (2.0 ** -121, 2.0 ** -120), (1e-37, 1e-37), (1e-38, 1e-38), (1e-38, 3e-39),
                                     (1e-40, 2e-40), (1e-43, 3e-43), (1e-45, 3e-45)])
def test_logits_as_small_as_the_temperature(vg, dtype, vocab, T, scale):
    g = torch.Generator().manual_seed(vocab)
    x = (randn(g, 3, vocab).double() * scale).to(dtype)
    x[1, ::3] = torch.finfo(dtype).min
    x[2, ::3] = -math.inf
    x[2, 1::3] = -1.0
    T = float(torch.tensor(T, dtype=torch.float32))
    u = torch.rand((3, 6), generator=g).to(DEV)
    check(vg, x, u, T=[T] * 3)
    check(vg, x, u, T=[T] * 3, k=[vocab // 3] * 3, p=[0.8] * 3)
    check(vg, x, u, T=[T] * 3, k=[3] * 3, mp=[0.05] * 3)


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("top", [1.0, -1.0, 2.0 ** 59, 2.0 ** 60, -2.0 ** 60, 1e30, 3e38, -3e38])
@pytest.mark.parametrize("T", [2.0 ** -119, 1e-38, 1e-45])
def test_large_logits_of_small_temperatures(vg, dtype, top, T):
    """Only the largest ones count, however near the next are."""
    x = torch.full((2, 4001), top, dtype=torch.float32, device=DEV).to(dtype)
    near = torch.nextafter(x[0, 0].cpu(), torch.tensor(-math.inf, dtype=dtype)).to(DEV)
    x[:, 3::2] = near
    x[1, 100:] = torch.finfo(dtype).min
    u = torch.rand((2, 6), generator=torch.Generator().manual_seed(1)).to(DEV)
    T = float(torch.tensor(T, dtype=torch.float32))
    check(vg, x, u, T=[T] * 2)
    check(vg, x, u, T=[T] * 2, k=[700] * 2, p=[0.9] * 2)
