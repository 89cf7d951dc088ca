"""Norms of heads with an eps that counts beside squares near the end of FP32's range and past it.  Tolerances: test_gpu_norm_rope's
(eps in FP32 is off by 2^-24 of itself, its inverse root by half of that, which the 1e-6 there has room for)."""
import pytest
import torch
from test_gpu_norm_rope import check
from test_gpu_verify_round import vg  # noqa: F401

pytestmark = pytest.mark.gpu

MOST = torch.finfo(torch.float32).max


@pytest.mark.parametrize("d,rot", [(128, 128), (128, 18), (16, 16), (256, 64), (16, 2)])
@pytest.mark.parametrize("eps", [1e30, 1e36, 1.2e37, 1e38, 3.2e38, MOST])
@pytest.mark.parametrize("scale", [1.0, 3e18, 1e19, 1.8e19, 1e20, 1e30])
def test_eps_beside_large_squares(vg, d, rot, eps, scale):
    check(vg, 8, 2, 3, 4, 2, d, rot, "half", torch.bfloat16, torch.bfloat16, 16, 3, eps=eps, scale=scale)


@pytest.mark.parametrize("rot", [64, 18])
@pytest.mark.parametrize("eps", [1e9, 1e30, MOST])
def test_eps_beside_fp16_heads(vg, rot, eps):
    check(vg, 9, 2, 3, 4, 2, 64, rot, "interleaved", torch.float16, torch.float16, 16, 3, eps=eps, scale=10000.0)
