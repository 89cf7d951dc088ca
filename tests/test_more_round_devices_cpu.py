"""The verify round's further calls on tensors of several devices: each is refused before anything is
launched.  No GPU is needed: the tensors have a device and a shape and no memory."""
from types import SimpleNamespace

import pytest
import torch
from test_verify_round_devices_cpu import HERE, THERE, V, B, cache, d, h, hq, n, vg  # noqa: F401
from torch._subclasses.fake_tensor import FakeTensorMode

pytestmark = pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.device_count() < 2,
                                reason="tensors of two devices need none or two")


def tensors(**where):
    """Every argument of the three calls on HERE, those named elsewhere."""
    i32, f32, f64, bf16 = torch.int32, torch.float32, torch.float64, torch.bfloat16
    shapes = dict(q=((B, n, hq, d), bf16), k=((B, n, h, d), bf16), v=((B, n, h, d), bf16), inv_freq=((d // 2,), f64),
                  lens=((B,), i32), depth=((B, n), i32), counts=((B,), i32), q_out=((B, n, hq, d), bf16),
                  q_weight=((d,), f32), k_weight=((d,), f32), prefix=((1,), i32), prefix_pages=((3,), i32),
                  tree=((B, n), torch.int64), out=((B, n, hq, d), bf16), lse=((B, n, hq), f32),
                  workspace=((1 << 20,), torch.uint8), logits=((4, V), f32), u=((4, 2), f32), temperature=((4,), f32),
                  top_k=((4,), i32), top_p=((4,), f32), min_p=((4,), f32), probs=((4, V), f32))
    with FakeTensorMode():
        t = {name: torch.empty(s, dtype=dt, device=where.get(name, HERE)) for name, (s, dt) in shapes.items()}
    return SimpleNamespace(**t)


def norms(vg, t, c, stream=None):
    return vg.qk_norm_rope_append(t.q, t.k, t.v, t.q_weight, t.k_weight, t.inv_freq, c, t.lens, t.depth, t.counts,
                                  q_out=t.q_out, stream=stream)


def attend(vg, t, c, stream=None):
    return vg.prefix_attention(t.q, c, t.lens, t.prefix, t.prefix_pages, t.tree, t.counts, out=t.out, lse=t.lse,
                               workspace=t.workspace, stream=stream)


def sample(vg, t, c, stream=None):
    return vg.sample(t.logits, t.u, t.temperature, t.top_k, t.top_p, t.min_p, t.probs, stream=stream)


@pytest.mark.parametrize("call,names", [
    (norms, ["k", "v", "q_weight", "k_weight", "inv_freq", "lens", "depth", "counts", "q_out"]),
    (attend, ["lens", "prefix", "prefix_pages", "tree", "counts", "out", "lse", "workspace"]),
    (sample, ["u", "temperature", "top_k", "top_p", "min_p", "probs"])])
def test_tensors_of_another_device_are_refused(vg, call, names):
    for name in names:
        with pytest.raises(ValueError, match="device"):
            call(vg, tensors(**{name: THERE}), cache(HERE))


@pytest.mark.parametrize("call", [norms, attend])
def test_a_cache_of_another_device_is_refused(vg, call):
    with pytest.raises(ValueError, match="device"):
        call(vg, tensors(), cache(THERE))


@pytest.mark.parametrize("call", [norms, attend, sample])
def test_a_stream_of_another_device_is_refused(vg, call):
    with pytest.raises(ValueError, match="device"):
        call(vg, tensors(), cache(HERE), stream=SimpleNamespace(device=THERE))


def test_a_workspace_for_a_cache_of_another_device_is_refused(vg):
    with pytest.raises(ValueError, match="device"):
        vg.prefix_attention_workspace(tensors().q, cache(THERE))
