"""The verify round's operators on the host: argument checks of the C ABI
(nothing is launched: fake addresses go in, and each call must come back with
its error), the cache descriptor's checks and the rotary frequencies."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from verify_gemm_gb300 import _lib, build

    build.build()
    _lib.load()
    return _lib


A = 0x10000        # an aligned fake address
ODD = 0x10001


def cache(L, **kw):
    c = L.vg_kv_cache()
    c.k, c.v, c.page_table = A, A, A
    c.type, c.heads, c.head_dim, c.page_size, c.pages = L.VG_TYPE_BF16, 2, 64, 16, 8
    for s in (c.k_stride, c.v_stride):
        s[0], s[1], s[2] = 16 * 128, 128, 64
    c.table_stride, c.batch, c.max_pages, c.k_scale, c.v_scale = 4, 3, 4, 1.0, 1.0
    for name, value in kw.items():
        if name.endswith("stride") and isinstance(value, tuple):
            getattr(c, name)[value[0]] = value[1]
        else:
            setattr(c, name, value)
    return c


def has_driver(L):
    """Whether the tensor maps can be encoded here (the driver's own function)."""
    c = cache(L)
    return L.vg_kv_cache_init(ctypes.byref(c)) == L.VG_OK


@pytest.mark.parametrize("status,kw", [
    (1, dict(k=None)), (1, dict(v=None)), (1, dict(page_table=None)), (1, dict(heads=0)),
    (1, dict(batch=0)), (1, dict(max_pages=0)), (1, dict(pages=0)), (1, dict(head_dim=0)),
    (1, dict(head_dim=24)), (1, dict(page_size=8)), (1, dict(page_size=17)), (1, dict(page_size=40)),
    (1, dict(table_stride=3)), (1, dict(type=2)), (1, dict(type=7)), (1, dict(k_scale=0.5)),
    (1, dict(v_scale=2.0)), (1, dict(k_stride=(1, 32))), (1, dict(v_stride=(2, 68))),
    (1, dict(type=3, k_scale=0.0)), (1, dict(type=3, v_scale=math.inf)),
    (1, dict(type=3, k_scale=math.nan)), (1, dict(type=3, k_stride=(1, 136))),
    (3, dict(head_dim=272, k_stride=(1, 1024))), (3, dict(pages=1 << 31)),
    (3, dict(max_pages=1 << 28, table_stride=1 << 28)), (3, dict(k_stride=(0, 1 << 40))),
    (2, dict(k=A + 8)), (2, dict(v=A + 2)),
])
def test_a_cache_is_refused(L, status, kw):
    base = dict(k_stride=(0, 1 << 20), v_stride=(0, 1 << 20)) if kw.get("head_dim", 0) > 256 else {}
    c = cache(L, **{**base, **kw})
    if kw.get("head_dim", 0) > 256:
        for s in (c.k_stride, c.v_stride):
            s[0], s[1], s[2] = 1 << 20, 1024, 512
    assert L.vg_kv_cache_init(ctypes.byref(c)) == status


def test_a_cache_that_was_not_prepared_or_has_changed_is_refused(L):
    c = cache(L)
    n = ctypes.c_size_t()
    assert L.vg_tree_attention_workspace_size(4, 2, ctypes.byref(c), ctypes.byref(n)) == 1
    assert L.vg_tree_attention_workspace_size(4, 2, None, ctypes.byref(n)) == 1
    d = L.vg_rope_desc()
    assert L.vg_rope_append(ctypes.byref(d), ctypes.byref(c), None) == 1
    assert L.vg_rope_append(None, None, None) == 1
    assert L.vg_kv_cache_init(None) == 1
    if not has_driver(L):
        pytest.skip("no driver here to encode a tensor map")
    assert L.vg_kv_cache_init(ctypes.byref(c)) == 0
    assert L.vg_tree_attention_workspace_size(4, 2, ctypes.byref(c), ctypes.byref(n)) == 0
    c.pages = 9
    assert L.vg_tree_attention_workspace_size(4, 2, ctypes.byref(c), ctypes.byref(n)) == 1


def test_probabilities_arguments(L):
    f = L.vg_probabilities
    assert f(None, 0, 1, 8, None, A, None) == 1
    assert f(A, 0, 1, 8, None, None, None) == 1
    assert f(A, 0, 0, 8, None, A, None) == 1
    assert f(A, 0, 1, 0, None, A, None) == 1
    assert f(A, 3, 1, 8, None, A, None) == 1
    assert f(A, -1, 1, 8, None, A, None) == 1
    assert f(A, 0, 1, 1 << 28, None, A, None) == 3
    assert f(A, 0, 1 << 27, 8, None, A, None) == 3
    assert f(ODD, 0, 1, 8, None, A, None) == 2
    assert f(A, 0, 1, 8, None, A + 8, None) == 2


def test_verify_arguments(L):
    def f(p=A, q=A, t=A, par=A, counts=None, u=A, B=2, n=4, rows=3, V=100, acc=A, path=A, out=A):
        return L.vg_verify_tree(p, q, t, par, counts, u, B, n, rows, V, acc, path, out, None)

    for kw in (dict(p=None), dict(q=None), dict(t=None), dict(par=None), dict(u=None), dict(acc=None),
               dict(path=None), dict(out=None), dict(B=0), dict(n=0), dict(rows=-1), dict(rows=5),
               dict(rows=0), dict(V=0)):
        assert f(**kw) == 1, kw
    assert f(n=1025) == 3 and f(V=1 << 28) == 3 and f(B=1 << 24) == 3
    assert f(p=A + 4) == 2 and f(q=A + 4) == 2


@pytest.mark.parametrize("rot,base,factor", [(64, 10000.0, 1.0), (128, 1e6, 8.0), (2, 500000.0, 4.0)])
def test_rope_frequencies(rot, base, factor):
    import verify_gemm_gb300 as vg

    plain = [base ** (-2.0 * j / rot) for j in range(rot // 2)]
    got, m = vg.rope_frequencies(rot, base, device="cpu")
    assert got.dtype == torch.float64 and m == 1.0
    # pow in 64 bits: a few units in the last place
    assert torch.allclose(got, torch.tensor(plain, dtype=torch.float64), rtol=1e-14, atol=0)
    lin, _ = vg.rope_frequencies(rot, base, "linear", factor, device="cpu")
    assert torch.allclose(lin * factor, got, rtol=1e-14, atol=0)
    if rot >= 4:
        ntk, _ = vg.rope_frequencies(rot, base, "ntk", factor, device="cpu")
        assert math.isclose(ntk[0], 1.0) and math.isclose(ntk[-1] * factor, got[-1], rel_tol=1e-12)
    y, m = vg.rope_frequencies(rot, base, "yarn", factor, context=32768, device="cpu")
    assert math.isclose(m, 0.1 * math.log(factor) + 1)
    for j, (a, b) in enumerate(zip(y.tolist(), plain)):
        turns = 32768 * b / (2 * math.pi)
        want = b if turns >= 32 else b / factor if turns <= 1 else None
        if want is not None:
            assert math.isclose(a, want, rel_tol=1e-12), j
        assert b / factor * (1 - 1e-12) <= a <= b * (1 + 1e-12)


def test_rope_frequencies_refuse():
    import verify_gemm_gb300 as vg

    for args in ((0,), (3,), (64, 1.0), (64, 1e4, "cubic"), (64, 1e4, "linear", 0.5),
                 (64, 1e4, "yarn", 2.0), (2, 1e4, "ntk", 2.0)):
        with pytest.raises(ValueError):
            vg.rope_frequencies(*args, device="cpu")
