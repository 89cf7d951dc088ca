"""The verify round's calls on tensors of several devices: each is refused before anything is
launched.  No GPU is needed: the tensors have a device and a shape and no memory.  (With one GPU a
tensor of a second cannot be made, not even so.)"""
from types import SimpleNamespace

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

pytestmark = pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.device_count() < 2,
                                reason="tensors of two devices need none or two")


@pytest.fixture(scope="module")
def vg():
    from verify_gemm_gb300 import _lib, build

    build.build()
    _lib.load_torch()
    import verify_gemm_gb300 as vg

    return vg


B, n, hq, h, d, V = 2, 3, 4, 2, 64, 50
HERE, THERE = torch.device("cuda", 1), torch.device("cuda", 0)


def tensors(**where):
    """Every argument of the four calls on HERE, those named elsewhere."""
    i32, f32, f64, bf16 = torch.int32, torch.float32, torch.float64, torch.bfloat16
    shapes = dict(q=((B, n, hq, d), bf16), k=((B, n, h, d), bf16), v=((B, n, h, d), bf16), inv_freq=((d // 2,), f64),
                  lens=((B,), i32), depth=((B, n), i32), counts=((B,), i32), q_out=((B, n, hq, d), bf16),
                  tree=((B, n), torch.int64), out=((B, n, hq, d), bf16), lse=((B, n, hq), f32),
                  workspace=((1 << 20,), torch.uint8), logits=((4, V), f32), temperature=((4,), f32), p_out=((4, V), f32),
                  p=((B, n, V), f32), pq=((B, n - 1, V), f32), tokens=((B, n), i32), parents=((B, n), i32), u=((B, n), f32))
    with FakeTensorMode():
        t = {name: torch.empty(s, dtype=dt, device=where.get(name, HERE)) for name, (s, dt) in shapes.items()}
    return SimpleNamespace(**t)


def cache(device):
    """What the calls ask of a cache, over addresses that are not read."""
    import ctypes

    from verify_gemm_gb300 import _lib as L

    c = L.vg_kv_cache()
    c.type, c.heads, c.head_dim, c.page_size, c.batch = L.VG_TYPE_BF16, h, d, 16, B
    return SimpleNamespace(_c=c, _at=ctypes.addressof(c), _device=device.index, k=SimpleNamespace(device=device), head_dim=d)


def rope(vg, t, c, stream=None):
    return vg.rope_append(t.q, t.k, t.v, t.inv_freq, c, t.lens, t.depth, t.counts, q_out=t.q_out, stream=stream)


def attend(vg, t, c, stream=None):
    return vg.tree_attention(t.q, c, t.lens, t.tree, t.counts, out=t.out, lse=t.lse, workspace=t.workspace, stream=stream)


def probabilities(vg, t, c, stream=None):
    return vg.probabilities(t.logits, t.temperature, t.p_out, stream=stream)


def verify(vg, t, c, stream=None):
    return vg.verify_tree(t.p, t.pq, t.tokens, t.parents, t.u, t.counts, stream=stream)


@pytest.mark.parametrize("call,names", [
    (rope, ["k", "v", "inv_freq", "lens", "depth", "counts", "q_out"]),
    (attend, ["lens", "tree", "counts", "out", "lse", "workspace"]),
    (probabilities, ["temperature", "p_out"]),
    (verify, ["pq", "tokens", "parents", "u", "counts"])])
def test_tensors_of_another_device_are_refused(vg, call, names):
    for name in names:
        with pytest.raises(ValueError, match="device"):
            call(vg, tensors(**{name: THERE}), cache(HERE))


@pytest.mark.parametrize("call", [rope, attend])
def test_a_cache_of_another_device_is_refused(vg, call):
    with pytest.raises(ValueError, match="device"):
        call(vg, tensors(), cache(THERE))


@pytest.mark.parametrize("call", [rope, attend, probabilities, verify])
def test_a_stream_of_another_device_is_refused(vg, call):
    with pytest.raises(ValueError, match="device"):
        call(vg, tensors(), cache(HERE), stream=SimpleNamespace(device=THERE))


def test_a_workspace_for_a_cache_of_another_device_is_refused(vg):
    with pytest.raises(ValueError, match="device"):
        vg.tree_attention_workspace(tensors().q, cache(THERE))
