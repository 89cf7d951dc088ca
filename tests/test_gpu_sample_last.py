"""A random number of 1 and more draws the last token that is kept, whatever it weighs."""
import math

import pytest
import torch
from test_gpu_verify_round import DEV, randn, vg  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("vocab", [2, 40, 5003, 151936, 300001])
@pytest.mark.parametrize("far", [1.0, 18.0, 24.0])
def test_last_token(vg, dtype, vocab, far):
    # the last one weighs e^-24 = 2^-34.6 at the least: more than the 2^-46 that a weight is rounded down to
    x = torch.full((3, vocab), -math.inf, dtype=dtype, device=DEV)
    x[:, 0] = 0
    x[0, -1] = -far
    x[1, vocab // 2] = -far
    x[2, 1:] = randn(torch.Generator().manual_seed(3), vocab - 1).mul(0.1).sub(far).to(dtype)
    u = torch.tensor([[1.0, 1.5, math.inf, 0.0]] * 3, device=DEV)
    for k, p in ((0, 1.0), (40, 1.0), (300, 1.0)):
        kk = torch.full((3,), k, dtype=torch.int32, device=DEV)
        out = torch.empty((3, vocab), device=DEV)
        got = vg.sample(x, u, top_k=kk, top_p=torch.full((3,), p, device=DEV), out=out).cpu()
        want = [int((row > 0).nonzero().max()) for row in out.cpu()]
        assert want[0] == vocab - 1 and want[1] == vocab // 2
        assert got.tolist() == [[w, w, w, 0] for w in want], (k, got.tolist(), want)
