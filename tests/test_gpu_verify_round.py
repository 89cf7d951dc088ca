"""Rotary append, tree attention, probabilities and draft verification
against plain 64-bit implementations, at the sizes and masks where they can
go wrong.

Tolerances.  u(T) = finfo(T).eps / 2 is the most a rounding to T is off,
relative to the value.
* Rotation: the angle reaches FP32 as a fraction of a turn, off by 2^-24 of
  at most half a turn, so by 2^-24 pi, and sincospif adds 2 units of 2^-23:
  together below 5e-7 on a cosine or sine; two products and a sum add 3 * 2^-24
  of |x1| + |x2|.  1e-6 (|x1| + |x2|) factor covers both; then u(T) |y|, or
  for E4M3 half a step: 2^-4 |y| or 2^-10 (the step of its subnormals is 2^-9).
* Attention: a score is a sum of d FP32 products, off by at most
  d 2^-24 sum |q k|; with the scaling and the exponential, a weight is off by
  e = 2 max(d 2^-24 scale sum |q k|) + 2^-20 relative.  The weights are rounded to
  T before they meet v (u(T) relative, and 2^-25 of the largest weight where
  FP16 runs out of normal numbers), so the output is off by at most
  (u(T) + 2 e) sum p |v| + 2^-25 sum |v| (FP16) + u(T) |o|.  With an 8-bit
  cache the same holds.  lse: e + 2^-20 (1 + |lse|).
* Probabilities: (x - max) / T and the exponential are off by |x - max| / T 2^-22
  + 2^-21 relative, the sum's additions by at most 2^-24 times their depth (under 2^7 steps).
* Verification gives whole numbers: equal.
"""
import math
from fractions import Fraction

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def vg():
    from verify_gemm_gb300 import build

    build.build()
    import verify_gemm_gb300 as vg

    torch.cuda.init()
    return vg


def u(dt):
    return torch.finfo(dt).eps / 2


def randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(DEV)


def build_cache(vg, g, B, slots, hkv, d, page, dtype, held, scales=(1.0, 1.0), fill="randn",
                heads_first=False, spare=3):
    """A cache with shuffled pages for `slots` slots of each sequence."""
    per = (slots + page - 1) // page
    total = B * per + spare
    table = torch.randperm(total, generator=g)[:B * per].reshape(B, per).to(torch.int32).to(DEV)
    shape = (total, hkv, page, d) if heads_first else (total, page, hkv, d)

    def one(scale):
        if fill == "nan":
            t = torch.full(shape, math.nan, dtype=torch.float32, device=DEV)
        else:
            t = randn(g, *shape, scale=1 / scale)
        t = t.to(held if held == E4M3 else dtype)
        return t.transpose(1, 2) if heads_first else t

    k, v = one(scales[0]), one(scales[1])
    return vg.KVCache(k, v, table, *scales), k, v, table


def slot_index(table, b, slots, page):
    s = torch.arange(slots, device=DEV)
    return table[b].long()[s // page], s % page


def some_tree(g, B, n):
    parents = torch.full((B, n), -1, dtype=torch.int32)
    depth = torch.zeros((B, n), dtype=torch.int32)
    words = [[1] for _ in range(B)]
    for b in range(B):
        for i in range(1, n):
            at = int(torch.randint(max(0, i - 4), i, (1,), generator=g))
            parents[b, i], depth[b, i] = at, depth[b, at] + 1
            words[b].append(words[b][at] | 1 << i)
    signed = [[w - (1 << 64) if w >> 63 else w for w in row] for row in words]
    return parents.to(DEV), depth.to(DEV), torch.tensor(signed, dtype=torch.int64).to(DEV)


# ------------------------------------------------------------------- rotation

def check_rope(vg, seed, B, n, hq, hkv, d, rot, layout, dtype, held, page, past, tree=False,
               counts=None, factor=1.0, strided=True, heads_first=False, in_place=False):
    g = torch.Generator().manual_seed(seed)
    scales = (0.03, 0.04) if held == E4M3 else (1.0, 1.0)
    lens = torch.tensor([past + 5 * b for b in range(B)], dtype=torch.int32)
    slots = int(lens.max()) + n
    cache, ck, cv, table = build_cache(vg, g, B, slots, hkv, d, page, dtype, held, scales,
                                       heads_first=heads_first)
    k0, v0 = ck.float().clone(), cv.float().clone()
    if strided:
        qkv = randn(g, B, n, hq + 2 * hkv, d, dtype=dtype)
        q, k, v = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
    else:
        q, k, v = (randn(g, B, n, h, d, dtype=dtype) for h in (hq, hkv, hkv))
    depth = some_tree(g, B, n)[1] if tree else None
    inv = (torch.rand(rot // 2, generator=g, dtype=torch.float64) ** 4).to(DEV)
    if rot:
        inv[0] = 1.0
    cnt = torch.tensor(counts, dtype=torch.int32).to(DEV) if counts is not None else None
    qref = q.double().clone()
    out = vg.rope_append(q, k, v, inv, cache, lens.to(DEV), depth=depth, counts=cnt, layout=layout,
                         factor=factor, q_out=q if in_place else None)
    if in_place:
        assert out.data_ptr() == q.data_ptr()
    pos = lens.to(DEV).long()[:, None] + (depth if depth is not None else torch.arange(n, device=DEV)).long()
    a = (pos[:, :, None].double() * inv)[:, :, None, :]
    i1, i2 = ((slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half"
              else (slice(0, rot, 2), slice(1, rot, 2)))

    def turned(x):
        y, e = x.clone(), torch.zeros_like(x)
        x1, x2 = x[..., i1], x[..., i2]
        y[..., i1] = (x1 * a.cos() - x2 * a.sin()) * factor
        y[..., i2] = (x1 * a.sin() + x2 * a.cos()) * factor
        e[..., i1] = e[..., i2] = 1e-6 * factor * (x1.abs() + x2.abs())
        return y, e

    want, e = turned(qref)
    used = torch.arange(n, device=DEV)[None, :] < (cnt[:, None] if cnt is not None else n)
    used = used.expand(B, n)
    want = torch.where(used[:, :, None, None], want, 0.0)
    assert ((out.double() - want).abs() <= e + u(dtype) * want.abs() + 1e-7).all()
    ky, ke = turned(k.double())
    vy, ve = v.double(), torch.zeros_like(v.double())
    wrote = torch.zeros(ck.shape[:2], dtype=torch.bool, device=DEV)
    for b in range(B):
        c = int(cnt[b]) if cnt is not None else n
        s = torch.arange(int(lens[b]), int(lens[b]) + c, device=DEV)
        at = table[b].long()[s // page], s % page
        wrote[at] = True
        for store, y, err, scale in ((ck, ky, ke, scales[0]), (cv, vy, ve, scales[1])):
            got, y, err = store[at].double(), y[b, :c] / scale, err[b, :c] / scale
            if held == E4M3:
                y = y.clamp(-448, 448)
                tol = err * (1 + 2 ** -4) + torch.maximum(2 ** -4 * y.abs(), torch.tensor(2.0 ** -10)) + 1e-6
            else:
                tol = err + u(dtype) * y.abs() + 1e-7
            assert ((got - y).abs() <= tol).all()
    # nothing else in the cache changed
    for store, before in ((ck, k0), (cv, v0)):
        assert torch.equal(store.float()[~wrote], before[~wrote])


@pytest.mark.parametrize("dtype,held", [(torch.bfloat16, None), (torch.float16, None),
                                        (torch.bfloat16, E4M3), (torch.float16, E4M3)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (128, 64), (80, 16), (96, 34), (256, 6), (16, 0)])
def test_rope_types_layouts_and_parts(vg, dtype, held, layout, d, rot):
    check_rope(vg, 1, 3, 5, 6, 2, d, rot, layout, dtype, held or dtype, 16, 13, tree=True,
               counts=[5, 2, 0], factor=1.25)


@pytest.mark.parametrize("B,n,hq,hkv", [(1, 1, 1, 1), (1, 1, 40, 40), (2, 1, 5, 5), (1, 300, 8, 1),
                                        (7, 9, 12, 4), (33, 3, 2, 2), (1, 2047, 6, 3)])
def test_rope_sizes(vg, B, n, hq, hkv):
    check_rope(vg, 2, B, n, hq, hkv, 128, 128, "half", torch.bfloat16, torch.bfloat16, 48, 31)


@pytest.mark.parametrize("strided,heads_first,in_place", [(False, False, False), (False, True, True),
                                                          (True, True, False)])
def test_rope_strides(vg, strided, heads_first, in_place):
    for layout, rot in (("half", 64), ("interleaved", 32), ("half", 18), ("interleaved", 22)):
        check_rope(vg, 3, 2, 6, 6, 3, 64, rot, layout, torch.float16, torch.float16, 32, 7,
                   strided=strided, heads_first=heads_first, in_place=in_place)


def test_rope_unaligned_inputs(vg):
    """Heads that begin between 16-byte borders."""
    g = torch.Generator().manual_seed(4)
    B, n, h, d = 2, 3, 2, 64
    cache, ck, cv, table = build_cache(vg, g, B, 16, h, d, 16, torch.bfloat16, torch.bfloat16)
    flat = randn(g, 3 * B * n * h * (d + 1) + 3, dtype=torch.bfloat16)
    views = [flat[1 + j * B * n * h * (d + 1):][:B * n * h * (d + 1)].view(B, n, h, d + 1)[..., :d]
             for j in range(3)]
    inv, m = vg.rope_frequencies(d, device=DEV)
    lens = torch.tensor([0, 9], dtype=torch.int32, device=DEV)
    got = vg.rope_append(*views, inv, cache, lens)
    k1, v1 = ck.clone(), cv.clone()
    want = vg.rope_append(*[x.contiguous() for x in views], inv, cache, lens)
    assert torch.equal(got, want) and torch.equal(k1, ck) and torch.equal(v1, cv)


@pytest.mark.parametrize("past", [100_000, 1_048_573, 2_000_000_000])
def test_rope_far_positions(vg, past):
    """The angle of a far position is as exact as that of a near one."""
    g = torch.Generator().manual_seed(5)
    d, n = 128, 4
    cache, *_ = build_cache(vg, g, 1, 16, 1, d, 16, torch.float16, torch.float16)
    q = torch.ones((1, n, 1, d), dtype=torch.float16, device=DEV)
    inv, _ = vg.rope_frequencies(d, 1e4, device=DEV)
    lens = torch.full((1,), past, dtype=torch.int32, device=DEV)
    out = vg.rope_append(q, q, q, inv, cache, lens)       # past the table: nothing is appended
    # angles with Python's whole numbers: position * inv as a fraction of 2 pi in 64 bits
    a = (past + torch.arange(n, dtype=torch.float64))[:, None] * inv.cpu()
    want = torch.cat((a.cos() - a.sin(), a.sin() + a.cos()), -1)
    # 64-bit reference: the product itself is off by 2^-53 of the angle
    tol = 2e-6 + u(torch.float16) * want.abs() + 4 * past * 2.0 ** -53
    assert ((out.double().cpu()[0, :, 0] - want).abs() <= tol).all()


@pytest.mark.parametrize("B,n,hq,hkv,d", [(3, 5001, 2, 1, 64), (77, 13, 4, 4, 64), (11, 333, 3, 1, 128)])
def test_rope_many_tokens_of_few_heads(vg, B, n, hq, hkv, d):
    """Blocks of several tokens, of more than one sequence, the last of them not full."""
    counts = [n - (7 * b) % n for b in range(B)]
    check_rope(vg, 7, B, n, hq, hkv, d, d, "half", torch.bfloat16, E4M3, 32, 3, counts=counts)
    check_rope(vg, 8, B, n, hq, hkv, d, 16, "interleaved", torch.float16, torch.float16, 16, 40)


def test_rope_any_frequency(vg):
    """Frequencies of either sign, of many turns a position, tiny ones and none."""
    inv = [0.0, -0.0, 1.0, -1.0, 0.3, -0.7, 2.0, 6.283185307179586, 12.5, 1e3 + 0.1, -123456.789, 1e-3, 1e-9,
           -1e-12, 2.0 ** -60, 2.0 ** -80, 1e-300, 5e-324, 2.0 ** 20, -2.0 ** 33, 3.14159, 1e6, 0.999999, -1e-6]
    d, n = 48, 5
    g = torch.Generator().manual_seed(9)
    cache, *_ = build_cache(vg, g, 1, 16, 1, d, 16, torch.float16, torch.float16)
    q = randn(g, 1, n, 1, d, dtype=torch.float16)
    f = torch.tensor(inv, dtype=torch.float64, device=DEV)
    lens = torch.full((1,), 1000, dtype=torch.int32, device=DEV)
    out = vg.rope_append(q, q, q, f, cache, lens).double().cpu()[0, :, 0]
    pos = (1000 + torch.arange(n, dtype=torch.float64))[:, None]
    a = pos * f.cpu()
    x1, x2 = q.double().cpu()[0, :, 0].split(d // 2, -1)
    want = torch.cat((x1 * a.cos() - x2 * a.sin(), x1 * a.sin() + x2 * a.cos()), -1)
    # the reference's product is off by 2^-53 of the angle, as is each of its values' argument
    size = torch.cat((x1.abs() + x2.abs(),) * 2, -1)
    tol = (2e-6 + 4 * a.abs().repeat(1, 2) * 2.0 ** -53) * size + u(torch.float16) * want.abs() + 2.0 ** -25
    assert ((out - want).abs() <= tol).all()


def test_rope_drops_what_has_no_page(vg):
    g = torch.Generator().manual_seed(6)
    B, n, h, d, page = 4, 20, 2, 64, 16
    cache, ck, cv, table = build_cache(vg, g, B, 32, h, d, page, torch.bfloat16, torch.bfloat16)
    table[1, 1] = -1
    table[2, 0] = ck.shape[0]
    lens = torch.tensor([20, 10, 0, -7], dtype=torch.int32, device=DEV)   # b 0 runs past the table
    x = randn(g, B, n, h, d, dtype=torch.bfloat16)
    k0 = ck.clone()
    out = vg.rope_append(x, x, x, torch.zeros(0, dtype=torch.float64, device=DEV), cache, lens)
    assert torch.equal(out, x)                               # rot 0: q passes as it is
    want = k0.clone()
    for b in range(B):
        for i in range(n):
            s = int(lens[b]) + i
            if 0 <= s < 32 and 0 <= int(table[b, s // page]) < ck.shape[0]:
                want[int(table[b, s // page]), s % page] = x[b, i]
    assert torch.equal(ck, want)


# ------------------------------------------------------------------ attention

def reference_attention(q, k, v, seen, scale):
    """q [r, d], k, v [s, d], seen [r, s] in 64 bits: (o, lse, sum p |v|, weight error, sum |v|)."""
    d = q.shape[1]
    x = (q @ torch.where(torch.isfinite(k), k, 0.0).T) * scale
    size = (q.abs() @ torch.where(torch.isfinite(k), k, 0.0).abs().T) * abs(scale)
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True) if x.shape[1] else torch.full((len(q), 1), -math.inf, device=DEV).double()
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.where(seen, torch.exp(x - top), 0.0)
    total = p.sum(-1, keepdim=True)
    vv = torch.where(torch.isfinite(v), v, 0.0)
    safe = torch.where(total == 0, 1.0, total)
    o, a = p @ vv / safe, p @ vv.abs() / safe
    most = torch.where(seen, size, 0.0).amax(-1, keepdim=True) if x.shape[1] else torch.zeros_like(total)
    e = 2 * most * d * 2.0 ** -24 + 2.0 ** -20
    return o, (top + torch.log(total))[:, 0], a, e, (seen.double() @ vv.abs())


def check_attention(vg, seed, B, n, hq, hkv, d, dtype, held, page, lens, counts=None, tree=None,
                    scale=None, fill="randn", heads_first=False, q_scale=1.0, poison=False,
                    workspace=None, break_pages=False, strided=False):
    g = torch.Generator().manual_seed(seed)
    scales = (0.03, 0.05) if held == E4M3 else (1.0, 1.0)
    slots = max(max(lens) + n, 1)
    cache, k, v, table = build_cache(vg, g, B, slots, hkv, d, page, dtype, held, scales,
                                     heads_first=heads_first)
    group = hq // hkv
    if strided:
        q = randn(g, B, hq, n, d + 16, dtype=dtype, scale=q_scale)[..., :d].transpose(1, 2)
    else:
        q = randn(g, B, n, hq, d, dtype=dtype, scale=q_scale)
    words = None
    if tree == "random":
        words = some_tree(g, B, n)[2]
    elif tree is not None:
        words = torch.tensor(tree, dtype=torch.int64).to(DEV)
    cnt = counts if counts is not None else [n] * B
    # everything that no row attends to is NaN or infinite
    owned = torch.zeros(k.shape[:2], dtype=torch.bool, device=DEV)
    for b in range(B):
        owned[slot_index(table, b, lens[b] + cnt[b], page)] = True
    if fill == "nan":
        for t in (k, v):
            bad = torch.full_like(t, math.nan)
            t.copy_(torch.where(owned[:, :, None, None], t.float(), bad.float()).to(t.dtype))
    if poison:
        # one drafted node of each sequence is not finite; some rows do not see it
        for b in range(B):
            at = slot_index(table, b, lens[b] + cnt[b], page)
            k.view(torch.uint8 if held == E4M3 else torch.int16)[at[0][-1], at[1][-1]] = 0x7F if held == E4M3 else 0x7FFF
            v.view(torch.uint8 if held == E4M3 else torch.int16)[at[0][-1], at[1][-1]] = 0x7F if held == E4M3 else 0x7FFF
    if break_pages:
        table[0, 0] = -1
        table[B - 1, -1] = k.shape[0] + 7
    lse = torch.full((B, n, hq), 7.0, dtype=torch.float32, device=DEV)
    out = torch.full((B, n, hq, d), 7.0, dtype=dtype, device=DEV)
    tl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    tc = torch.tensor(counts, dtype=torch.int32, device=DEV) if counts is not None else None
    ws = workspace if workspace is not None else vg.tree_attention_workspace(q, cache)
    got = vg.tree_attention(q, cache, tl, tree=words, counts=tc, scale=scale, out=out, lse=lse,
                            workspace=ws)
    assert got.data_ptr() == out.data_ptr()
    again, lse2 = torch.empty_like(out), torch.empty_like(lse)
    vg.tree_attention(q, cache, tl, tree=words, counts=tc, scale=scale, out=again, lse=lse2, workspace=ws)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))     # the same bits each time
    assert torch.equal(lse.view(torch.int32), lse2.view(torch.int32))
    sc = d ** -0.5 if scale is None else scale
    for b in range(B):
        total = lens[b] + cnt[b]
        at = slot_index(table.clamp(0, k.shape[0] - 1), b, total, page)
        seen = torch.ones((n, total), dtype=torch.bool, device=DEV)
        for i in range(n):
            word = int(words[b, i]) & (2 ** 64 - 1) if words is not None else (1 << (i + 1)) - 1
            for j in range(cnt[b]):
                seen[i, lens[b] + j] = bool(word >> j & 1)
            if i >= cnt[b]:
                seen[i] = False
        s = torch.arange(total, device=DEV)
        there = table[b].long()[s // page]
        seen &= ((there >= 0) & (there < k.shape[0]))[None, :]
        for h in range(hkv):
            kk, vv = (t[at[0], at[1], h].double() * c for t, c in ((k, scales[0]), (v, scales[1])))
            rows = q[b, :, h * group:(h + 1) * group].double().reshape(n * group, d)
            see = seen[:, None, :].expand(n, group, total).reshape(n * group, total)
            o, ls, a, e, av = reference_attention(rows, kk, vv, see, sc)
            y = out[b, :, h * group:(h + 1) * group].double().reshape(n * group, d)
            l2 = lse[b, :, h * group:(h + 1) * group].double().reshape(-1)
            bad = ~torch.isfinite(vv).all() and (see[:, ~torch.isfinite(vv).all(-1)].any(-1))
            good = ~bad if torch.is_tensor(bad) else torch.ones(n * group, dtype=torch.bool, device=DEV)
            empty = ~see.any(-1) if total else torch.ones(n * group, dtype=torch.bool, device=DEV)
            assert (y[empty] == 0).all() and (l2[empty] == -math.inf).all()
            tol = (u(dtype) + 2 * e) * a + u(dtype) * o.abs() + 1e-7
            if dtype == torch.float16:
                tol = tol + 2.0 ** -25 * av
            ok = good & ~empty
            assert ((y - o).abs() <= tol)[ok].all(), (b, h, ((y - o).abs() / tol)[ok].max())
            assert ((l2 - ls).abs() <= e[:, 0] + 2.0 ** -20 * (1 + ls.abs()))[ok].all()
            assert torch.isnan(y[~good & ~empty]).all()
    return ws


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 129, 1000]


@pytest.mark.parametrize("dtype,held", [(torch.bfloat16, None), (torch.float16, None),
                                        (torch.bfloat16, E4M3), (torch.float16, E4M3)])
@pytest.mark.parametrize("d", [16, 64, 80, 96, 128, 144, 192, 256])
def test_attention_types_and_head_sizes(vg, dtype, held, d):
    check_attention(vg, 11, len(LENS), 4, 6, 2, d, dtype, held or dtype, 16, LENS, fill="nan")


@pytest.mark.parametrize("n,hq,hkv", [(1, 1, 1), (1, 8, 1), (1, 16, 1), (1, 17, 1), (2, 40, 40),
                                      (3, 5, 1), (8, 8, 8), (8, 10, 2), (16, 8, 2), (16, 8, 1),
                                      (17, 10, 2), (33, 4, 1), (64, 4, 4), (64, 16, 2), (61, 24, 3)])
def test_attention_rows(vg, n, hq, hkv):
    """Rows per shared head from 1 to 512."""
    for dtype, held in ((torch.bfloat16, torch.bfloat16), (torch.float16, E4M3)):
        check_attention(vg, 12, 3, n, hq, hkv, 128, dtype, held, 64, [200, 0, 77], tree="random",
                        counts=[n, max(1, n - 1), (n + 1) // 2], fill="nan")


@pytest.mark.parametrize("page", [16, 32, 48, 80, 128, 2048])
def test_attention_pages(vg, page):
    for heads_first in (False, True):
        check_attention(vg, 13, 4, 5, 4, 2, 64, torch.bfloat16, torch.bfloat16, page, [0, 47, 333, 1300],
                        heads_first=heads_first, fill="nan")


def test_attention_strided_q_and_scale(vg):
    check_attention(vg, 14, 2, 7, 6, 3, 96, torch.bfloat16, torch.bfloat16, 32, [90, 31], scale=0.3,
                    strided=True)


def test_attention_large_scores(vg):
    """Scores in the hundreds: one key takes all, the running maximum matters."""
    for dtype in (torch.bfloat16, torch.float16):
        check_attention(vg, 15, 2, 3, 8, 2, 128, dtype, dtype, 16, [700, 40], q_scale=60.0)


def test_attention_masks_that_leave_nothing(vg):
    """Nodes that attend to no draft, with and without a prefix."""
    tree = [[0, 0b10, 0b101, 0], [0, 0, 0b1, 0b1111], [-1, -1, -1, -1]]
    check_attention(vg, 16, 3, 4, 4, 2, 64, torch.bfloat16, torch.bfloat16, 16, [0, 33, 0],
                    tree=tree, counts=[4, 3, 0], fill="nan")


@pytest.mark.parametrize("held", [None, E4M3])
@pytest.mark.parametrize("n,hq", [(6, 2), (40, 8)])
def test_attention_ignores_what_it_does_not_attend_to(vg, held, n, hq):
    """The last node is NaN: rows that see it are NaN, the others as if it were not there."""
    chain = [[(1 << (i + 1)) - 1 for i in range(n)] for _ in range(2)]
    check_attention(vg, 17, 2, n, hq, 2, 128, torch.bfloat16, held or torch.bfloat16, 16, [100, 5],
                    tree=chain, poison=True, fill="nan")


def test_attention_missing_pages(vg):
    check_attention(vg, 18, 3, 4, 4, 2, 64, torch.bfloat16, torch.bfloat16, 16, [100, 60, 120],
                    break_pages=True)


@pytest.mark.parametrize("length,B,n,hq,hkv", [(20011, 1, 1, 8, 1), (5003, 2, 8, 10, 5),
                                               (30000, 1, 64, 8, 1), (3001, 20, 2, 16, 8)])
def test_attention_long_and_ragged(vg, length, B, n, hq, hkv):
    lens = [max(0, length - 977 * b * b % (length + 1)) for b in range(B)]
    check_attention(vg, 19, B, n, hq, hkv, 128, torch.bfloat16, torch.bfloat16, 64, lens, tree="random")


def test_attention_one_workspace_for_calls_in_turn(vg):
    """Calls of several shapes on one workspace, which every call leaves as it found it."""
    ws = None
    for seed, (B, n, hq, hkv, lens) in enumerate([(1, 8, 40, 40, [3000]), (3, 1, 16, 2, [5000, 1, 700]),
                                                  (1, 64, 8, 1, [4000]), (1, 8, 40, 40, [900])]):
        if ws is None:
            g = torch.Generator().manual_seed(0)
            cache, *_ = build_cache(vg, g, 1, 16, 1, 128, 16, torch.bfloat16, torch.bfloat16)
            big = torch.empty((1, 64, 64, 128), dtype=torch.bfloat16, device=DEV)
            ws = vg.tree_attention_workspace(big, cache)
        check_attention(vg, 20 + seed, B, n, hq, hkv, 128, torch.bfloat16, torch.bfloat16, 64, lens,
                        workspace=ws)
    from verify_gemm_gb300 import workspace_error
    assert workspace_error(ws) == 0


def test_attention_offsets_past_32_bits(vg):
    """Pages whose elements lie beyond 2^32 elements (8 GB) from the start."""
    d, page, hkv = 128, 64, 2
    pages = (1 << 32) // (page * hkv * d) + 8
    k = torch.empty((pages, page, hkv, d), dtype=torch.bfloat16, device=DEV)
    v = torch.empty((pages, page, hkv, d), dtype=torch.bfloat16, device=DEV)
    table = torch.tensor([[pages - 1, 0, pages - 3]], dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(31)
    for p in table[0].tolist():
        k[p], v[p] = randn(g, page, hkv, d), randn(g, page, hkv, d)
    cache = vg.KVCache(k, v, table)
    x = randn(g, 1, 8, hkv, d, dtype=torch.bfloat16)
    lens = torch.tensor([150], dtype=torch.int32, device=DEV)
    vg.rope_append(x, x, x, torch.zeros(0, dtype=torch.float64, device=DEV), cache, lens)
    assert torch.equal(k[pages - 3, 22:30], x[0])
    near = vg.KVCache(k[table[0].long()].contiguous(), v[table[0].long()].contiguous(),
                      torch.arange(3, dtype=torch.int32, device=DEV)[None])
    assert torch.equal(vg.tree_attention(x, cache, lens), vg.tree_attention(x, near, lens))


# -------------------------------------------------------------- probabilities

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (2, 2), (3, 7), (1, 1000), (5, 4097), (2, 50257),
                                        (3, 151936), (1, 300001), (200, 1023)])
def test_probabilities(vg, dtype, rows, vocab):
    g = torch.Generator().manual_seed(rows + vocab)
    x = randn(g, rows, vocab, dtype=dtype, scale=3.0)
    t = (0.3 + torch.rand(rows, generator=g)).to(DEV)
    t[0] = 1.0
    if rows > 2:
        t[1], t[2] = 0.0, 100.0
    got = vg.probabilities(x, temperature=t).double()
    xd = x.double()
    z = (xd - xd.amax(-1, keepdim=True)) / torch.where(t > 0, t, 1.0).double()[:, None]
    want = torch.softmax(z, -1)
    first = (xd == xd.amax(-1, keepdim=True)).to(torch.int8).argmax(-1)
    hot = torch.zeros_like(want).scatter_(1, first[:, None], 1.0)
    want = torch.where((t > 0)[:, None], want, hot)
    tol = want * (z.abs() * 2.0 ** -22 + 2.0 ** -21 + 2.0 ** -17) + 1e-37
    assert ((got - want).abs() <= tol).all()
    if rows > 2:
        assert torch.equal(got[1], hot[1])
    assert torch.equal(vg.probabilities(x[:1], None), vg.probabilities(x[:1], t[:1]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_probabilities_at_every_share_of_a_row(vg, dtype):
    """Vocabularies whose share of a block takes every multiple of 4 KB of its shared
    memory, up to those that do not fit: each against a sum in 64 bits."""
    g = torch.Generator().manual_seed(3)
    for vocab in list(range(9000, 420000, 15361)) + [98000, 98304, 190000, 196607, 393000, 786432, 800011]:
        x = randn(g, 2, vocab, dtype=dtype, scale=2.0)
        y = vg.probabilities(x).double()
        want = torch.softmax(x.double(), -1)
        assert ((y - want).abs() <= want * (2.0 ** -16 + 40 * 2.0 ** -22) + 1e-37).all(), vocab


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_probabilities_of_masked_rows(vg, dtype):
    low = torch.finfo(dtype).min
    V = 5003
    x = torch.zeros((8, V), dtype=dtype, device=DEV)
    x[0] = -math.inf                                   # nothing left
    x[1] = low                                         # all at the lowest value
    x[2, 1:] = -math.inf                               # one left
    x[3, 5:] = low
    x[4, 7] = math.nan
    x[5, 9] = math.inf
    x[6] = -math.inf
    x[7] = 1.0                                         # ties
    t = torch.tensor([1, 1, 1, 1, 1, 1, 0, 0], dtype=torch.float32, device=DEV)
    y = vg.probabilities(x, temperature=t)
    assert (y[0] == 0).all() and (y[6] == 0).all()
    assert torch.allclose(y[1], torch.full((V,), 1 / V, device=DEV), rtol=1e-5)
    assert y[2, 0] == 1 and (y[2, 1:] == 0).all()
    assert torch.allclose(y[3, :5], torch.full((5,), 0.2, device=DEV), rtol=1e-6) and (y[3, 5:] == 0).all()
    assert torch.isnan(y[4]).all() and torch.isnan(y[5]).all()
    assert y[7, 0] == 1 and (y[7, 1:] == 0).all()      # the lowest index
    small = torch.full((2, 9), low, dtype=dtype, device=DEV)
    z = vg.probabilities(small, temperature=torch.tensor([0.0, 1.0], device=DEV))
    assert z[0, 0] == 1 and (z[0, 1:] == 0).all() and torch.allclose(z[1], torch.full((9,), 1 / 9, device=DEV))


# --------------------------------------------------------------- verification

def reference_verify(p, q, tokens, parents, u, count):
    """The rule in exact fractions, the residual kept as a distribution."""
    n, V = len(p), len(p[0])
    F = [[Fraction(float(x)) for x in row] for row in p.tolist()]
    Q = [[Fraction(float(x)) for x in row] for row in q.tolist()]
    cur, r, S, path, out = 0, F[0], Fraction(1), [], []
    for i in range(1, count):
        f, t = int(parents[i]), int(tokens[i])
        if f != cur or f >= i or f >= len(Q) or not 0 <= t < V:
            continue
        if Fraction(float(u[i])) * Q[cur][t] * S < r[t]:
            path.append(i)
            out.append(t)
            cur, r, S = i, F[i], Fraction(1)
        else:
            r = [max(a - S * b, Fraction(0)) for a, b in zip(r, Q[cur])]
            S = sum(r)
    if sum(r) == 0:
        r = F[cur]
    whole, run, last = sum(r), Fraction(0), -1
    for k, x in enumerate(r):
        run += x
        if run > Fraction(float(u[0])) * whole:
            last = k
            break
    return len(path), path + [-1] * (n - len(path)), out + [last] + [-1] * (n - len(out))


def draw_round(g, B, n, V, sharp, agree, tree, rows=None):
    rows = rows or (n if tree else max(n - 1, 1))
    base = torch.randn((B, n, V), generator=g) * sharp
    p = torch.softmax(base, -1)
    q = torch.softmax(base[:, :rows] + torch.randn((B, rows, V), generator=g) * agree, -1)
    parents = torch.full((B, n), -1, dtype=torch.int32)
    tokens = torch.full((B, n), -1, dtype=torch.int32)
    for b in range(B):
        for i in range(1, n):
            f = int(torch.randint(max(0, min(i, rows) - 3), min(i, rows), (1,), generator=g)) if tree else i - 1
            parents[b, i] = f
            tokens[b, i] = int(torch.multinomial(q[b, min(f, rows - 1)], 1, generator=g))
    u = torch.rand((B, n), generator=g)
    return p, q, tokens, parents, u


def check_verify(vg, p, q, tokens, parents, u, counts=None):
    B, n, V = p.shape
    c = torch.tensor(counts, dtype=torch.int32).to(DEV) if counts is not None else None
    acc, path, out = vg.verify_tree(p.to(DEV), q.to(DEV), tokens.to(DEV), parents.to(DEV), u.to(DEV), counts=c)
    taken = 0
    for b in range(B):
        want = reference_verify(p[b], q[b], tokens[b], parents[b], u[b], counts[b] if counts else n)
        assert (int(acc[b]), path[b].tolist(), out[b].tolist()) == want, b
        taken += want[0]
    return taken


@pytest.mark.parametrize("n,V,tree", [(1, 5, False), (2, 1, False), (2, 3, False), (4, 33, False),
                                      (8, 257, False), (6, 31, True), (16, 64, True), (33, 100, True),
                                      (5, 1025, True), (3, 2050, True)])
def test_verify(vg, n, V, tree):
    g = torch.Generator().manual_seed(n * 1000 + V)
    for agree in (0.1, 1.0, 3.0):
        p, q, tokens, parents, u = draw_round(g, 6, n, V, 2.0, agree, tree)
        check_verify(vg, p, q, tokens, parents, u)
        check_verify(vg, p, q, tokens, parents, u, counts=[n, max(1, n // 2), 1, 0, n, n])


def test_verify_greedy_rows(vg):
    """One-hot targets: a draft holds where it is the target's token."""
    g = torch.Generator().manual_seed(7)
    B, n, V = 12, 5, 50
    p = torch.zeros((B, n, V)).scatter_(2, torch.randint(0, 3, (B, n, 1), generator=g), 1.0)
    q = torch.softmax(torch.randn((B, n - 1, V), generator=g), -1)
    tokens = torch.randint(0, 3, (B, n), generator=g, dtype=torch.int32)
    parents = torch.arange(-1, n - 1, dtype=torch.int32).expand(B, n).contiguous()
    acc = check_verify(vg, p, q, tokens, parents, torch.rand((B, n), generator=g))
    assert 0 < acc < B * (n - 1)


def test_verify_many_siblings_and_equal_rows(vg):
    g = torch.Generator().manual_seed(8)
    B, n, V = 8, 40, 60
    p, q, tokens, parents, u = draw_round(g, B, n, V, 1.0, 2.0, True)
    parents[:, 1:] = 0                                  # all drafted from the root
    u[:] = u * 0.2 + 0.79                               # mostly refused
    tokens[:, 1:] = torch.multinomial(q[:, 0], n - 1, replacement=True, generator=g).to(torch.int32)
    check_verify(vg, p, q, tokens, parents, u)
    # disjoint p and q: every child is refused and the residual stays p
    p2, q2 = torch.zeros_like(p), torch.zeros_like(q)
    p2[:, :, 30:], q2[:, :, :30] = 1 / 32, 1 / 32
    tokens[:, 1:] = torch.randint(0, 30, (B, n - 1), generator=g, dtype=torch.int32)
    assert check_verify(vg, p2, q2, tokens, parents, u) == 0
    # q = p: always accepted; and q > p everywhere: the residual is empty and p is drawn from
    assert check_verify(vg, p, p, tokens, parents, u * 0.9) == B
    tokens[:, 1:] = 0
    check_verify(vg, p, (p * 1.5).clamp(max=1), tokens, parents, torch.full_like(u, 0.97))
    # a row of zeros has no token
    acc, path, out = vg.verify_tree(*(t.to(DEV) for t in (torch.zeros_like(p), q, tokens, parents, u)))
    assert (acc == 0).all() and (out == -1).all() and (path == -1).all()


def test_verify_passes_over_nodes_that_fit_nowhere(vg):
    g = torch.Generator().manual_seed(9)
    B, n, V = 6, 8, 40
    p, q, tokens, parents, u = draw_round(g, B, n, V, 1.5, 0.3, False, rows=5)
    tokens[0, 1], tokens[1, 2], parents[2, 3], parents[3, 1] = V, -5, 3, 100
    parents[4, 2], parents[5, 1] = -9, 1
    check_verify(vg, p, q, tokens, parents, u)


def test_verify_wide_rows_and_odd_vocabularies(vg):
    """Rows of a real vocabulary against running sums in 64 bits."""
    for V, n, tree in ((151936, 4, False), (151937, 6, True), (32003, 12, True)):
        g = torch.Generator().manual_seed(V)
        p, q, tokens, parents, u = (t.to(DEV) for t in draw_round(g, 3, n, V, 2.5, 1.5, tree))
        acc, path, out = vg.verify_tree(p, q, tokens, parents, u)
        for b in range(3):
            cur, r, S, kept = 0, p[b, 0].double(), 1.0, []
            for i in range(1, n):
                if int(parents[b, i]) != cur:
                    continue
                t = int(tokens[b, i])
                if float(u[b, i]) * float(q[b, cur, t]) * S < float(r[t]):
                    kept.append(i)
                    cur, r, S = i, p[b, i].double(), 1.0
                else:
                    r = (r - S * q[b, cur].double()).clamp(min=0)
                    S = float(r.sum())
            run = r.cumsum(0)
            last = int((run <= float(u[b, 0]) * run[-1]).sum())
            assert int(acc[b]) == len(kept) and path[b].tolist() == kept + [-1] * (n - len(kept))
            assert out[b].tolist() == [int(tokens[b, i]) for i in kept] + [last] + [-1] * (n - len(kept))


def test_verify_edges_of_the_random_numbers(vg):
    p = torch.tensor([[[0.25, 0.0, 0.25, 0.5]]])
    q = torch.zeros((1, 1, 4))
    t = torch.full((1, 1), -1, dtype=torch.int32)
    for x, want in ((0.0, 0), (0.2499, 0), (0.25, 2), (0.4999, 2), (0.5, 3), (1 - 2.0 ** -24, 3), (1.0, 3),
                    (-1.0, 0), (2.0 ** -40, 0)):
        _, _, out = vg.verify_tree(p.to(DEV), q.to(DEV), t.to(DEV), t.to(DEV), torch.tensor([[x]], device=DEV))
        assert out[0].tolist() == [want, -1], x


def test_verify_keeps_the_targets_distribution(vg):
    """The first token that comes out is distributed as p, whatever q is: 20000
    rounds, each frequency within 5 standard deviations."""
    g = torch.Generator().manual_seed(10)
    B, n, V = 20000, 4, 6
    p1 = torch.softmax(torch.randn((n, V), generator=g) * 1.2, -1)
    q1 = torch.softmax(torch.randn((n, V), generator=g) * 1.2, -1)
    parents = torch.tensor([-1, 0, 0, 1], dtype=torch.int32).expand(B, n).contiguous()
    tokens = torch.full((B, n), -1, dtype=torch.int32)
    for i, f in ((1, 0), (2, 0), (3, 1)):
        tokens[:, i] = torch.multinomial(q1[f], B, replacement=True, generator=g).to(torch.int32)
    u = torch.rand((B, n), generator=g)
    _, _, out = vg.verify_tree(p1.expand(B, n, V).contiguous().to(DEV), q1.expand(B, n, V).contiguous().to(DEV),
                               tokens.to(DEV), parents.to(DEV), u.to(DEV))
    got = torch.bincount(out[:, 0].cpu().long(), minlength=V).double() / B
    want = p1[0].double()
    assert ((got - want).abs() <= 5 * (want * (1 - want) / B).sqrt()).all()


# ------------------------------------------------- graphs, streams, refusals

def test_a_captured_round_follows_the_device_words(vg):
    """Rotation, attention and verification captured once, replayed at other lengths."""
    g = torch.Generator().manual_seed(12)
    B, n, h, d, V = 2, 5, 4, 64, 500
    cache, ck, cv, table = build_cache(vg, g, B, 2000, 2, d, 64, torch.bfloat16, torch.bfloat16)
    q, k, v = randn(g, B, n, h, d, dtype=torch.bfloat16), *(randn(g, B, n, 2, d, dtype=torch.bfloat16) for _ in "kv")
    inv, _ = vg.rope_frequencies(d, device=DEV)
    lens = torch.tensor([10, 20], dtype=torch.int32, device=DEV)
    x = randn(g, B * n, V, dtype=torch.bfloat16)
    qd = torch.softmax(randn(g, B, n, V), -1)
    tokens = torch.randint(0, V, (B, n), generator=g, dtype=torch.int32).to(DEV)
    parents = torch.arange(-1, n - 1, dtype=torch.int32).expand(B, n).contiguous().to(DEV)
    uu = torch.rand((B, n), generator=g).to(DEV)
    ws = vg.tree_attention_workspace(q, cache)

    def step():
        o = vg.tree_attention(vg.rope_append(q, k, v, inv, cache, lens), cache, lens, workspace=ws)
        return o, vg.verify_tree(vg.probabilities(x).view(B, n, V), qd, tokens, parents, uu)

    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        o, ver = step()
    for now in ((10, 20), (1900, 0), (64, 1333)):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got, gv = o.clone(), [t.clone() for t in ver]
        o2, v2 = step()
        assert torch.equal(got, o2) and all(torch.equal(a, b) for a, b in zip(gv, v2))


def test_work_runs_on_the_given_stream(vg):
    g = torch.Generator().manual_seed(13)
    x = randn(g, 4, 70001, dtype=torch.bfloat16)
    want = vg.probabilities(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(want)
    vg.probabilities(x, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)


def test_what_a_call_makes_belongs_to_its_stream(vg):
    """The outputs and the workspace that a call is not given are made on the stream that it is
    given: a current stream that is held up delays none of it."""
    g = torch.Generator().manual_seed(15)
    cache, ck, cv, table = build_cache(vg, g, 2, 5000, 2, 128, 16, torch.bfloat16, torch.bfloat16)
    q = randn(g, 2, 8, 4, 128, dtype=torch.bfloat16)
    lens = torch.tensor([4900, 17], dtype=torch.int32, device=DEV)
    logits = randn(g, 3, 5001)
    p = torch.softmax(randn(g, 2, 4, 999), -1).contiguous()
    tokens = torch.zeros((2, 4), dtype=torch.int32, device=DEV)
    parents = torch.arange(-1, 3, dtype=torch.int32, device=DEV).expand(2, 4).contiguous()
    rnd = torch.full((2, 4), 0.5, device=DEV)

    def calls(stream):
        return [vg.tree_attention(q, cache, lens, stream=stream), vg.probabilities(logits, stream=stream),
                *vg.verify_tree(p, p, tokens, parents, rnd, stream=stream)]

    want = calls(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(400_000_000)                       # some 0.2 s
    held = torch.cuda.Event()
    held.record()
    got = calls(side)
    side.synchronize()
    early = not held.query()
    torch.cuda.synchronize()
    assert early
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals(vg):
    g = torch.Generator().manual_seed(14)
    cache, ck, cv, table = build_cache(vg, g, 2, 64, 2, 64, 16, torch.bfloat16, torch.bfloat16)
    q = randn(g, 2, 3, 4, 64, dtype=torch.bfloat16)
    k = randn(g, 2, 3, 2, 64, dtype=torch.bfloat16)
    lens = torch.zeros(2, dtype=torch.int32, device=DEV)
    inv, _ = vg.rope_frequencies(64, device=DEV)
    for bad in (lambda: vg.KVCache(ck.float(), cv.float(), table),
                lambda: vg.KVCache(ck, cv.half(), table),
                lambda: vg.KVCache(ck, cv, table.long()),
                lambda: vg.KVCache(ck[..., :24], cv[..., :24], table),
                lambda: vg.KVCache(ck[:, :15], cv[:, :15], table),
                lambda: vg.KVCache(ck, cv, table, 0.5),
                lambda: vg.KVCache(ck.cpu(), cv.cpu(), table),
                lambda: vg.rope_append(q, k, k, inv, cache, lens.long()),
                lambda: vg.rope_append(q, k, k, inv.float(), cache, lens),
                lambda: vg.rope_append(q, k, k, inv, cache, lens, layout="other"),
                lambda: vg.rope_append(q, k[:1], k, inv, cache, lens),
                lambda: vg.rope_append(q.half(), k.half(), k.half(), inv, cache, lens),
                lambda: vg.rope_append(q, k, k, torch.cat((inv, inv)), cache, lens),
                lambda: vg.rope_append(q, k, k, inv, cache, lens, depth=lens),
                lambda: vg.tree_attention(q[:, :, :3], cache, lens),
                lambda: vg.tree_attention(q.half(), cache, lens),
                lambda: vg.tree_attention(q, cache, lens[:1]),
                lambda: vg.tree_attention(q, cache, lens, tree=lens),
                lambda: vg.tree_attention(q, cache, lens, scale=math.inf),
                lambda: vg.tree_attention(randn(g, 2, 65, 4, 64, dtype=torch.bfloat16), cache, lens),
                lambda: vg.tree_attention(q, cache, lens, lse=torch.empty(3, device=DEV)),
                lambda: vg.tree_attention(q, cache, lens, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV)),
                lambda: vg.probabilities(torch.zeros((2, 4), device=DEV).t()),
                lambda: vg.probabilities(torch.zeros((2, 4), dtype=torch.float64, device=DEV)),
                lambda: vg.probabilities(torch.zeros((2, 4), device=DEV), temperature=torch.ones(3, device=DEV)),
                lambda: vg.probabilities(torch.zeros(8)),
                lambda: vg.verify_tree(torch.zeros((2, 3, 4), device=DEV), None, lens, lens, lens)):
        with pytest.raises((ValueError, vg.VGError)):
            bad()


def test_a_row_without_numbers_stays_without(vg):
    """A query of NaN gives NaN, and leaves the other rows alone."""
    g = torch.Generator().manual_seed(15)
    for n, hq in ((3, 2), (20, 4)):
        cache, ck, cv, table = build_cache(vg, g, 1, 300, 2, 64, 16, torch.bfloat16, torch.bfloat16)
        q = randn(g, 1, n, hq, 64, dtype=torch.bfloat16)
        lens = torch.tensor([200], dtype=torch.int32, device=DEV)
        want = vg.tree_attention(q, cache, lens)
        q[0, 1, 0] = math.nan
        lse = torch.empty((1, n, hq), device=DEV)
        got = vg.tree_attention(q, cache, lens, lse=lse)
        assert torch.isnan(got[0, 1, 0]).all() and torch.isnan(lse[0, 1, 0])
        got[0, 1, 0], want[0, 1, 0] = 0, 0
        assert torch.equal(got, want)


@pytest.mark.parametrize("n,hq,hkv,d", [(16, 4, 1, 128), (64, 8, 2, 64), (50, 6, 1, 96), (64, 16, 1, 128),
                                        (12, 24, 4, 80)])
@pytest.mark.parametrize("dtype,held", [(torch.bfloat16, None), (torch.float16, None), (torch.bfloat16, E4M3)])
def test_attention_many_rows(vg, n, hq, hkv, d, dtype, held):
    """More than 32 rows a cache head, at lengths about the tiles' borders, with nodes that
    are not finite where some rows do not see them."""
    lens = [0, 1, 127, 128, 129, 255, 1100, 40]
    check_attention(vg, 41, len(lens), n, hq, hkv, d, dtype, held or dtype, 16, lens, fill="nan", tree="random",
                    counts=[n, 1, n // 2, n, n, 0, n, n - 1])
    chain = [[(1 << (i + 1)) - 1 if i < 63 else -1 for i in range(n)] for _ in lens]
    check_attention(vg, 42, len(lens), n, hq, hkv, d, dtype, held or dtype, 16, lens, fill="nan", tree=chain,
                    poison=True)


@pytest.mark.parametrize("n,hq,d,length", [(26, 8, 128, 20601), (64, 2, 64, 9001), (20, 8, 192, 9001),
                                           (8, 2, 256, 12345), (1, 1, 128, 30000)])
@pytest.mark.parametrize("held", [torch.bfloat16, E4M3])
def test_attention_of_few_units_over_long_caches(vg, n, hq, d, length, held):
    """Units that most of the device's blocks have a part in."""
    check_attention(vg, 47, 1, n, hq, 1, d, torch.bfloat16, held, 64, [length], tree="random")
    check_attention(vg, 48, 3, n, hq, 1, d, torch.bfloat16, held, 16, [length // 2, 0, length], counts=[n, 1, n])


@pytest.mark.parametrize("n,hq,d", [(9, 4, 192), (13, 5, 144), (16, 5, 256), (40, 1, 176), (64, 3, 192), (7, 3, 128)])
@pytest.mark.parametrize("dtype,held", [(torch.bfloat16, None), (torch.float16, None), (torch.bfloat16, E4M3)])
def test_attention_rows_that_fill_no_block(vg, n, hq, d, dtype, held):
    check_attention(vg, 51, 3, n, hq, 1, d, dtype, held or dtype, 32, [700, 3, 131], tree="random")
    check_attention(vg, 52, 2, n, hq, 1, d, dtype, held or dtype, 48, [90, 260], counts=[n // 2, n], poison=True)


@pytest.mark.parametrize("n,hq,hkv,d", [(2, 40, 40, 96), (3, 10, 5, 64), (5, 20, 5, 128), (1, 7, 7, 256)])
@pytest.mark.parametrize("dtype,held", [(torch.bfloat16, None), (torch.float16, E4M3)])
def test_attention_of_many_short_sequences(vg, n, hq, hkv, d, dtype, held):
    """Units of one tile among longer ones, several to a block."""
    lens = [2, 0, 61, 64, 65, 1, 200, 5, 7, 30, 1000, 59, 62, 3, 3, 3, 4, 17, 48]
    check_attention(vg, 53, len(lens), n, hq, hkv, d, dtype, held or dtype, 16, lens, tree="random")
    check_attention(vg, 54, len(lens), n, hq, hkv, d, dtype, held or dtype, 32, lens[::-1], poison=True)


def test_attention_negative_and_zero_scale(vg):
    for n, hq in ((4, 4), (40, 4)):
        for scale in (-0.2, 0.0):
            check_attention(vg, 43, 2, n, hq, 2, 128, torch.bfloat16, torch.bfloat16, 16, [300, 9], scale=scale)


def test_the_example_runs(vg):
    import runpy
    import os
    from conftest import ROOT
    runpy.run_path(os.path.join(ROOT, "examples", "verify_round.py"), run_name="__main__")
