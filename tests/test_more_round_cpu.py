"""The verify round's further operators on the host: argument checks of the C ABI.  Nothing is
launched: fake addresses go in, and each call must come back with its error."""
import ctypes
import math
import struct

import pytest
from test_verify_round_cpu import A, L, cache  # noqa: F401


def prepared(L):
    """A cache as vg_kv_cache_init leaves it, but for the tensor maps, for which it takes a driver: the
    mark over its fields."""
    c, h, m = cache(L), 0xcbf29ce484222325, (1 << 64) - 1

    def bits(x):
        return struct.unpack("<I", struct.pack("<f", x))[0]

    words = [c.k, c.v, c.page_table, c.type | c.heads << 32, c.head_dim | c.page_size << 32, c.pages]
    for i in range(3):
        words += [c.k_stride[i], c.v_stride[i]]
    words += [c.table_stride, c.batch | c.max_pages << 32, bits(c.k_scale) | bits(c.v_scale) << 32]
    for w in words:
        h = (h ^ w) * 0x100000001b3 & m
        h ^= h >> 29
    c.opaque[32] = h | 1
    n = ctypes.c_size_t()
    assert L.vg_prefix_attention_workspace_size(65, 2, ctypes.byref(c), ctypes.byref(n)) == 1
    assert L.vg_prefix_attention_workspace_size(4, 2 * 4097, ctypes.byref(c), ctypes.byref(n)) == 3   # past the mark
    return c


def rope(L, **kw):
    d = L.vg_qk_norm_rope_desc()
    r = d.rope
    r.q = r.k = r.v = r.q_out = r.inv_freq = r.lens = A
    for s in (r.q_stride, r.k_stride, r.v_stride):
        s[0], s[1], s[2] = 512, 128, 64
    r.type, r.layout, r.n, r.q_heads, r.rot, r.factor = L.VG_TYPE_BF16, L.VG_ROPE_HALF, 4, 2, 64, 1.0
    d.q_weight = d.k_weight = A
    d.weight_type, d.eps = L.VG_TYPE_FP32, 1e-6
    for name, value in kw.items():
        setattr(d if hasattr(d, name) else r, name, value)
    return d


@pytest.mark.parametrize("status,kw", [
    (1, dict(q=None)), (1, dict(k=None)), (1, dict(v=None)), (1, dict(q_out=None)), (1, dict(lens=None)),
    (1, dict(inv_freq=None)), (1, dict(n=0)), (1, dict(q_heads=0)), (1, dict(rot=3)), (1, dict(rot=-2)),
    (1, dict(rot=66)), (1, dict(type=2)), (1, dict(type=1)), (1, dict(layout=2)), (2, dict(q=A + 1)),
    (1, dict(eps=0.0)), (1, dict(eps=-1e-6)), (1, dict(eps=math.inf)), (1, dict(eps=math.nan)), (1, dict(eps=1e-39)),
    (1, dict(weight_type=1)), (1, dict(weight_type=3)), (1, dict(weight_type=-1)), (2, dict(q_weight=A + 2)),
    (2, dict(k_weight=A + 1, weight_type=0)), (3, dict(n=1 << 30)),
])
def test_norms_are_refused(L, status, kw):
    c = cache(L)
    assert L.vg_qk_norm_rope_append(ctypes.byref(rope(L)), ctypes.byref(c), None) == 1      # not prepared
    assert L.vg_qk_norm_rope_append(None, ctypes.byref(c), None) == 1
    assert L.vg_qk_norm_rope_append(ctypes.byref(rope(L)), None, None) == 1
    c = prepared(L)
    assert L.vg_qk_norm_rope_append(ctypes.byref(rope(L, **kw)), ctypes.byref(c), None) == status


def attention(L, **kw):
    d = L.vg_attention_desc()
    d.q = d.out = d.lens = A
    d.q_stride[0], d.q_stride[1], d.q_stride[2] = 512, 128, 64
    d.type, d.n, d.q_heads, d.scale = L.VG_TYPE_BF16, 4, 2, 0.125
    for name, value in kw.items():
        setattr(d, name, value)
    return d


@pytest.mark.parametrize("status,kw,args", [
    (1, dict(q=None), {}), (1, dict(out=None), {}), (1, dict(lens=None), {}), (1, dict(n=0), {}), (1, dict(n=65), {}),
    (1, dict(q_heads=3), {}), (1, dict(q_heads=0), {}), (1, dict(type=2), {}), (1, dict(type=1), {}),
    (1, dict(scale=math.inf), {}), (1, dict(scale=math.nan), {}), (2, dict(q=A + 8), {}), (2, dict(out=A + 2), {}),
    (1, {}, dict(prefix=None)), (1, {}, dict(pages=None)), (1, {}, dict(most=-1)), (2, {}, dict(prefix=A + 2)),
    (2, {}, dict(pages=A + 1)), (3, {}, dict(most=1 << 28)), (3, dict(q_heads=2 * 4097), {}),
])
def test_prefix_attention_is_refused(L, status, kw, args):
    c = cache(L)
    n = ctypes.c_size_t()

    def call(d, prefix=A, pages=A, most=4):
        return L.vg_prefix_attention(ctypes.byref(d), ctypes.byref(c), prefix, pages, most, A, 1 << 30, None)

    assert call(attention(L)) == 1                                                           # not prepared
    assert L.vg_prefix_attention(None, ctypes.byref(c), A, A, 4, A, 1 << 30, None) == 1
    assert L.vg_prefix_attention_workspace_size(4, 2, ctypes.byref(c), ctypes.byref(n)) == 1
    assert L.vg_prefix_attention_workspace_size(4, 2, None, ctypes.byref(n)) == 1
    c = prepared(L)
    assert L.vg_prefix_attention_workspace_size(65, 2, ctypes.byref(c), ctypes.byref(n)) == 1
    assert L.vg_prefix_attention_workspace_size(4, 2, ctypes.byref(c), None) == 1
    assert call(attention(L, **kw), **args) == status


@pytest.mark.parametrize("status,kw", [
    (1, dict(x=None)), (1, dict(u=None)), (1, dict(tokens=None)), (1, dict(rows=0)), (1, dict(rows=-4)),
    (1, dict(vocab=0)), (1, dict(draws=0)), (1, dict(row_stride=99)), (1, dict(type=3)), (1, dict(type=-1)),
    (2, dict(x=A + 1)), (2, dict(x=A + 2, type=2)), (2, dict(out=A + 2)), (2, dict(u=A + 2)), (2, dict(tokens=A + 1)),
    (2, dict(temperature=A + 2)), (2, dict(top_k=A + 1)), (2, dict(top_p=A + 3)), (2, dict(min_p=A + 2)),
    (3, dict(vocab=1 << 28, row_stride=1 << 28)), (3, dict(rows=1 << 26)), (3, dict(draws=65537)),
    (3, dict(row_stride=1 << 39)),
])
def test_draws_are_refused(L, status, kw):
    d = L.vg_sample_desc()
    d.x = d.u = d.tokens = A
    d.rows, d.vocab, d.row_stride, d.type, d.draws = 3, 100, 128, 0, 1
    for name, value in kw.items():
        setattr(d, name, value)
    assert L.vg_sample(ctypes.byref(d), None) == status
    assert L.vg_sample(None, None) == 1
