"""Norms of the heads of q and k with the rotation and the append, against 64 bits.

Tolerances.  u(T) = finfo(T).eps / 2 is the most a rounding to T is off, relative
to the value.  A sum of at most 256 squares in FP32, 16 or fewer of them in
a row and the rest in a tree, is off by at most 2^-24 * 24 relative, its inverse root
by half of that and 2^-22 of rsqrt's own, and two products add 2^-23: a normed
element is off by less than 1e-6 of itself.  The rotation adds 1e-6 (|x1| + |x2|) as
in rope_append (the angle's 2^-24 pi, sincospif, two products and a sum).  Then
u(T) |y|, or for E4M3 half a step: 2^-4 |y| or 2^-10.
"""
import math

import pytest
import torch
from test_gpu_verify_round import DEV, E4M3, build_cache, randn, some_tree, u, vg  # noqa: F401

pytestmark = pytest.mark.gpu


def normed(x, w, eps):
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return y * w.double() if w is not None else y


def check(vg, seed, B, n, hq, hkv, d, rot, layout, dtype, held, page, past, tree=False, counts=None, factor=1.0,
          eps=1e-6, weights="same", strided=True, in_place=False, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    scales = (0.03, 0.04) if held == E4M3 else (1.0, 1.0)
    lens = torch.tensor([past + 5 * b for b in range(B)], dtype=torch.int32)
    cache, ck, cv, table = build_cache(vg, g, B, int(lens.max()) + n, hkv, d, page, dtype, held, scales)
    k0, v0 = ck.float().clone(), cv.float().clone()
    if strided:
        qkv = randn(g, B, n, hq + 2 * hkv, d, dtype=dtype, scale=scale)
        q, k, v = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
    else:
        q, k, v = (randn(g, B, n, h, d, dtype=dtype, scale=scale) for h in (hq, hkv, hkv))
    depth = some_tree(g, B, n)[1] if tree else None
    inv = (torch.rand(rot // 2, generator=g, dtype=torch.float64) ** 4).to(DEV)
    wt = {"same": dtype, "fp32": torch.float32, "none": None}[weights]
    wq, wk = ((1 + randn(g, d, scale=0.3)).to(wt) if wt is not None else None for _ in "qk")
    cnt = torch.tensor(counts, dtype=torch.int32).to(DEV) if counts is not None else None
    want_q, want_k, want_v = normed(q, wq, eps), normed(k, wk, eps), v.double().clone()
    out = vg.qk_norm_rope_append(q, k, v, wq, wk, inv, cache, lens.to(DEV), depth=depth, counts=cnt, eps=eps,
                                 layout=layout, factor=factor, q_out=q if in_place else None)
    if in_place:
        assert out.data_ptr() == q.data_ptr()
    pos = lens.to(DEV).long()[:, None] + (depth if depth is not None else torch.arange(n, device=DEV)).long()
    a = (pos[:, :, None].double() * inv)[:, :, None, :]
    i1, i2 = ((slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half"
              else (slice(0, rot, 2), slice(1, rot, 2)))

    def turned(x):
        y, e = x.clone(), 1e-6 * x.abs()
        x1, x2 = x[..., i1], x[..., i2]
        y[..., i1] = (x1 * a.cos() - x2 * a.sin()) * factor
        y[..., i2] = (x1 * a.sin() + x2 * a.cos()) * factor
        e[..., i1] = e[..., i2] = 2e-6 * factor * (x1.abs() + x2.abs())
        return y, e

    want, e = turned(want_q)
    used = (torch.arange(n, device=DEV)[None, :] < (cnt[:, None] if cnt is not None else n)).expand(B, n)
    want = torch.where(used[:, :, None, None], want, 0.0)
    assert ((out.double() - want).abs() <= e + u(dtype) * want.abs() + 1e-7).all()
    ky, ke = turned(want_k)
    wrote = torch.zeros(ck.shape[:2], dtype=torch.bool, device=DEV)
    for b in range(B):
        c = int(cnt[b]) if cnt is not None else n
        s = torch.arange(int(lens[b]), int(lens[b]) + c, device=DEV)
        at = table[b].long()[s // page], s % page
        wrote[at] = True
        for store, y, err, sc in ((ck, ky, ke, scales[0]), (cv, want_v, torch.zeros_like(want_v), scales[1])):
            got, y, err = store[at].double(), y[b, :c] / sc, err[b, :c] / sc
            if held == E4M3:
                y = y.clamp(-448, 448)
                tol = err * (1 + 2 ** -4) + torch.maximum(2 ** -4 * y.abs(), torch.tensor(2.0 ** -10)) + 1e-6
            else:
                tol = err + u(dtype) * y.abs() + 1e-7
            assert ((got - y).abs() <= tol).all()
    for store, before in ((ck, k0), (cv, v0)):
        assert torch.equal(store.float()[~wrote], before[~wrote])


@pytest.mark.parametrize("dtype,held", [(torch.bfloat16, None), (torch.float16, None),
                                        (torch.bfloat16, E4M3), (torch.float16, E4M3)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (128, 64), (80, 16), (80, 80), (96, 34), (240, 112),
                                   (256, 256), (256, 6), (16, 16), (16, 0), (32, 16)])
def test_types_layouts_and_parts(vg, dtype, held, layout, d, rot):
    check(vg, 1, 3, 5, 6, 2, d, rot, layout, dtype, held or dtype, 16, 13, tree=True, counts=[5, 2, 0], factor=1.25,
          weights=("same", "fp32", "none")[(d + rot) // 16 % 3])


@pytest.mark.parametrize("B,n,hq,hkv", [(1, 1, 1, 1), (1, 1, 40, 40), (2, 1, 5, 5), (1, 300, 8, 1), (7, 9, 12, 4),
                                        (33, 3, 2, 2), (1, 2047, 6, 3), (1, 1, 320, 8), (1, 20000, 2, 1)])
def test_sizes(vg, B, n, hq, hkv):
    check(vg, 2, B, n, hq, hkv, 128, 128, "half", torch.bfloat16, torch.bfloat16, 48, 31)


@pytest.mark.parametrize("strided,in_place", [(False, False), (False, True), (True, False)])
@pytest.mark.parametrize("layout,rot", [("half", 64), ("interleaved", 32), ("half", 18), ("interleaved", 22)])
def test_strides_and_in_place(vg, strided, in_place, layout, rot):
    check(vg, 3, 2, 6, 6, 3, 64, rot, layout, torch.float16, torch.float16, 32, 7, strided=strided, in_place=in_place)


@pytest.mark.parametrize("eps", [1e-30, 1e-5, 1.0])
def test_eps(vg, eps):
    check(vg, 4, 2, 3, 4, 2, 128, 64, "half", torch.bfloat16, torch.bfloat16, 16, 3, eps=eps)
    check(vg, 5, 2, 3, 4, 2, 96, 18, "half", torch.float16, torch.float16, 16, 3, eps=eps)


@pytest.mark.parametrize("rot", [128, 18])
def test_heads_whose_squares_pass_the_range(vg, rot):
    """BF16 heads up to 3e38: their squares are not FP32 numbers.  And tiny ones, beside eps."""
    for scale in (1e30, 1e37, 3e18, 1e-20, 1e-38):
        check(vg, 6, 2, 3, 4, 2, 128, rot, "half", torch.bfloat16, torch.bfloat16, 16, 3, scale=scale)


def test_unaligned_inputs(vg):
    """Heads that begin between 16-byte borders give what aligned ones do, but for the sums' order."""
    g = torch.Generator().manual_seed(4)
    B, n, h, d = 2, 3, 2, 64
    cache, ck, cv, table = build_cache(vg, g, B, 16, h, d, 16, torch.float16, torch.float16)
    flat = randn(g, 3 * B * n * h * (d + 1) + 3, dtype=torch.float16)
    views = [flat[1 + j * B * n * h * (d + 1):][:B * n * h * (d + 1)].view(B, n, h, d + 1)[..., :d] for j in range(3)]
    inv, m = vg.rope_frequencies(d, device=DEV)
    lens = torch.tensor([0, 9], dtype=torch.int32, device=DEV)
    w = torch.ones(d, device=DEV)
    got = vg.qk_norm_rope_append(*views, w, w, inv, cache, lens)
    k1, v1 = ck.clone(), cv.clone()
    want = vg.qk_norm_rope_append(*[x.contiguous() for x in views], w, w, inv, cache, lens)
    # two roundings of values that differ by 4e-6 (|x1| + |x2|) at most
    for a, b in ((got, want), (k1, ck)):
        a, b = a.double(), b.double()
        assert ((a - b).abs() <= 2 * u(torch.float16) * b.abs() + 4e-6 * 8).all()
    assert torch.equal(v1, cv)


def test_zero_rows_and_rows_without_numbers(vg):
    """A head of zeros stays one; a NaN stays within its head, and so does an infinity."""
    g = torch.Generator().manual_seed(7)
    for rot in (64, 18):
        cache, ck, cv, table = build_cache(vg, g, 1, 16, 2, 64, 16, torch.bfloat16, torch.bfloat16)
        q, k, v = (randn(g, 1, 4, h, 64, dtype=torch.bfloat16) for h in (3, 2, 2))
        inv = torch.ones(rot // 2, dtype=torch.float64, device=DEV)
        lens = torch.zeros(1, dtype=torch.int32, device=DEV)
        w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
        want = vg.qk_norm_rope_append(q, k, v, w, w, inv, cache, lens)
        q2 = q.clone()
        q2[0, 0, 1], q2[0, 1, 0, 5], q2[0, 2, 2, 63] = 0, math.nan, math.inf
        got = vg.qk_norm_rope_append(q2, k, v, w, w, inv, cache, lens)
        assert (got[0, 0, 1] == 0).all() and torch.isnan(got[0, 1, 0]).all() and torch.isnan(got[0, 2, 2, 63])
        assert (got[0, 2, 2, rot:63] == 0).all()
        for i, h in ((0, 1), (1, 0), (2, 2)):
            got[0, i, h] = want[0, i, h] = 0
        assert torch.equal(got, want)


def test_drops_what_has_no_page(vg):
    g = torch.Generator().manual_seed(6)
    B, n, h, d, page = 4, 20, 2, 64, 16
    for rot in (0, 10):
        cache, ck, cv, table = build_cache(vg, g, B, 32, h, d, page, torch.bfloat16, torch.bfloat16)
        table[1, 1] = -1
        table[2, 0] = ck.shape[0]
        lens = torch.tensor([20, 10, 0, -7], dtype=torch.int32, device=DEV)   # b 0 runs past the table
        x = randn(g, B, n, h, d, dtype=torch.bfloat16)
        v0 = cv.clone()
        vg.qk_norm_rope_append(x, x, x, None, None, torch.zeros(rot // 2, dtype=torch.float64, device=DEV), cache, lens)
        for b in range(B):
            for i in range(n):
                s = int(lens[b]) + i
                if 0 <= s < 32 and 0 <= int(table[b, s // page]) < ck.shape[0]:
                    v0[int(table[b, s // page]), s % page] = x[b, i]
        assert torch.equal(cv, v0)


def test_refusals(vg):
    g = torch.Generator().manual_seed(14)
    cache, ck, cv, table = build_cache(vg, g, 2, 64, 2, 64, 16, torch.bfloat16, torch.bfloat16)
    q, k = randn(g, 2, 3, 4, 64, dtype=torch.bfloat16), randn(g, 2, 3, 2, 64, dtype=torch.bfloat16)
    lens = torch.zeros(2, dtype=torch.int32, device=DEV)
    inv, _ = vg.rope_frequencies(64, device=DEV)
    w = torch.ones(64, device=DEV)

    def call(q=q, k=k, v=k, wq=w, wk=w, inv=inv, lens=lens, **kw):
        return vg.qk_norm_rope_append(q, k, v, wq, wk, inv, cache, lens, **kw)

    call()
    for kw in (dict(wq=w[:63]), dict(wk=w.double()), dict(wq=w.half()), dict(wq=w.bfloat16()), dict(wk=w.cpu()),
               dict(wq=torch.ones(128, device=DEV)[::2]), dict(wq=torch.ones((1, 64), device=DEV)),
               dict(eps=0.0), dict(eps=-1.0), dict(eps=math.inf), dict(eps=math.nan), dict(eps=1e-40),
               dict(layout="other"), dict(lens=lens.long()), dict(k=k[:1]), dict(inv=inv.float()),
               dict(q=q.half(), k=k.half(), v=k.half())):
        with pytest.raises((ValueError, vg.VGError)):
            call(**kw)
