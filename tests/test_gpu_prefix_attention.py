"""Tree attention behind a shared prefix, against 64 bits over each sequence's whole cache.

Tolerances: those of tree attention (a weight is off by e = 2 max(d 2^-24 scale
sum |q k|) + 2^-20 relative; the output by (u(T) + 2 e) sum p |v| + 2^-25 sum |v|
(FP16 products) + u(T) |o|; lse by e + 2^-20 (1 + |lse|)).  Joining the two parts takes two
exponentials of differences, a division and a sum, each within 2^-22: less
than the 2^-20 that e has beside the scores' own error.
"""
import math

import pytest
import torch
from test_gpu_verify_round import (DEV, E4M3, randn, reference_attention, some_tree, u,  # noqa: F401
                                   vg)

pytestmark = pytest.mark.gpu


def build(vg, g, B, hkv, d, page, dtype, held, prefix, lens, n, scales, heads_first=False):
    """A cache whose first pages are the prefix's, and pages of each sequence's own behind them.  The
    row of a sequence that shares names no page before; one that is shorter has all its own."""
    whole = prefix // page
    ends = [(x + n + page - 1) // page for x in lens]
    width = max(max(ends), 1)
    total = whole + sum(ends) + 2
    order = torch.randperm(total, generator=g).to(torch.int32)
    pages, at = order[:whole], whole
    table = torch.full((B, width), -1, dtype=torch.int32)
    for b in range(B):
        first = whole if lens[b] >= whole * page else 0
        for i in range(first, ends[b]):
            table[b, i] = order[at]
            at += 1
    shape = (total, hkv, page, d) if heads_first else (total, page, hkv, d)

    def one(scale):
        t = randn(g, *shape, scale=1 / scale).to(held if held == E4M3 else dtype)
        return t.transpose(1, 2) if heads_first else t

    k, v, table = one(scales[0]), one(scales[1]), table.to(DEV)
    return vg.KVCache(k, v, table, *scales), k, v, table, pages.to(DEV)


def check(vg, seed, B, n, hq, hkv, d, dtype, held, page, prefix, own, counts=None, tree=None, scale=None,
          strided=False, heads_first=False, poison=False, break_pages=False, q_scale=1.0, limit=None, workspace=None):
    g = torch.Generator().manual_seed(seed)
    scales = (0.03, 0.05) if held == E4M3 else (1.0, 1.0)
    lens = [max(0, prefix + x) for x in own]
    cache, k, v, table, pages = build(vg, g, B, hkv, d, page, dtype, held, prefix, lens, n, scales, heads_first)
    if strided:
        q = randn(g, B, hq, n, d + 16, dtype=dtype, scale=q_scale)[..., :d].transpose(1, 2)
    else:
        q = randn(g, B, n, hq, d, dtype=dtype, scale=q_scale)
    whole = prefix // page
    words = some_tree(g, B, n)[2] if tree == "random" else torch.tensor(tree, dtype=torch.int64).to(DEV) if tree else None
    cnt = counts if counts is not None else [n] * B
    path = [[int(pages[i]) if lens[b] >= whole * page and i < whole else int(table[b, i]) if i < table.shape[1] else -1
             for i in range(max(whole, table.shape[1]))] for b in range(B)]
    if poison:                                           # all that nobody attends to is NaN, in the prefix, too
        code = 0x7F if held == E4M3 else 0x7FFF
        owned = torch.zeros(k.shape[:2], dtype=torch.bool)
        for b in range(B):
            for s in range(lens[b] + cnt[b]):
                owned[path[b][s // page], s % page] = True
        for t in (k, v):
            raw = t.view(torch.uint8 if held == E4M3 else torch.int16)
            raw.copy_(torch.where(owned.to(DEV)[:, :, None, None], raw, torch.full_like(raw, code)))
    if break_pages:
        pages[0] = -1
        pages[-1] = k.shape[0] + 3
        for b in range(B):
            if lens[b] >= whole * page:
                path[b][0] = path[b][whole - 1] = -1
    tl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    tc = torch.tensor(counts, dtype=torch.int32, device=DEV) if counts is not None else None
    tp = torch.tensor([prefix], dtype=torch.int32, device=DEV)
    out = torch.full((B, n, hq, d), 7.0, dtype=dtype, device=DEV)
    lse = torch.full((B, n, hq), 7.0, dtype=torch.float32, device=DEV)
    ws = workspace if workspace is not None else vg.prefix_attention_workspace(q, cache)
    got = vg.prefix_attention(q, cache, tl, tp, pages, tree=words, counts=tc, scale=scale, out=out, lse=lse, workspace=ws)
    assert got.data_ptr() == out.data_ptr()
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    vg.prefix_attention(q, cache, tl, tp, pages, tree=words, counts=tc, scale=scale, out=out2, lse=lse2, workspace=ws)
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16))       # the same bits each time
    assert torch.equal(lse.view(torch.int32), lse2.view(torch.int32))
    assert vg.workspace_error(ws) == 0
    sc, group = d ** -0.5 if scale is None else scale, hq // hkv
    for b in range(B):
        total = lens[b] + cnt[b]
        s = torch.arange(total, device=DEV)
        there = torch.tensor(path[b] + [-1], device=DEV)[s // page] if total else s
        ok_page = (there >= 0) & (there < k.shape[0])
        at = there.clamp(0, k.shape[0] - 1), s % page
        seen = torch.ones((n, total), dtype=torch.bool, device=DEV)
        for i in range(n):
            word = int(words[b, i]) & (2 ** 64 - 1) if words is not None else (1 << (i + 1)) - 1
            for j in range(cnt[b]):
                seen[i, lens[b] + j] = bool(word >> j & 1)
            if i >= cnt[b]:
                seen[i] = False
        seen &= ok_page[None, :]
        for h in range(hkv):
            kk, vv = (t[at[0], at[1], h].double() * c for t, c in ((k, scales[0]), (v, scales[1])))
            rows = q[b, :, h * group:(h + 1) * group].double().reshape(n * group, d)
            see = seen[:, None, :].expand(n, group, total).reshape(n * group, total)
            o, ls, a, e, av = reference_attention(rows, kk, vv, see, sc)
            y = out[b, :, h * group:(h + 1) * group].double().reshape(n * group, d)
            l2 = lse[b, :, h * group:(h + 1) * group].double().reshape(-1)
            empty = ~see.any(-1) if total else torch.ones(n * group, dtype=torch.bool, device=DEV)
            assert (y[empty] == 0).all() and (l2[empty] == -math.inf).all()
            tol = (u(dtype) + 2 * e) * a + u(dtype) * o.abs() + 1e-7
            if dtype == torch.float16:
                tol = tol + 2.0 ** -25 * av
            assert ((y - o).abs() <= tol)[~empty].all(), (b, h, ((y - o).abs() / tol)[~empty].max())
            assert ((l2 - ls).abs() <= e[:, 0] + 2.0 ** -20 * (1 + ls.abs()))[~empty].all()


# sequences that begin right behind the prefix, some that do not have all of it
OWN = [0, 1, 15, 16, 130, 77, -1, -200, 700, -5000]


@pytest.mark.parametrize("dtype,held", [(torch.bfloat16, None), (torch.float16, None),
                                        (torch.bfloat16, E4M3), (torch.float16, E4M3)])
@pytest.mark.parametrize("d", [16, 64, 80, 128, 144, 192, 256])
def test_types_and_head_sizes(vg, dtype, held, d):
    check(vg, 11, len(OWN), 3, 6, 2, d, dtype, held or dtype, 16, 403, OWN, poison=True)


@pytest.mark.parametrize("B,n,hq,hkv", [(1, 1, 1, 1), (2, 1, 8, 8), (16, 1, 2, 1), (17, 1, 1, 1), (5, 8, 10, 2),
                                        (9, 16, 4, 1), (3, 64, 8, 2), (33, 4, 8, 1), (70, 2, 16, 1), (2, 61, 24, 3)])
def test_rows(vg, B, n, hq, hkv):
    """From one row a cache head to two thousand over the prefix, and 1 to 512 over the rest."""
    own = [(37 * b) % 300 for b in range(B)]
    for dtype, held in ((torch.bfloat16, torch.bfloat16), (torch.float16, E4M3)):
        check(vg, 12, B, n, hq, hkv, 128, dtype, held, 64, 1000, own, tree="random",
              counts=[max(0, n - b % 3) for b in range(B)])


@pytest.mark.parametrize("page", [16, 48, 128, 2048])
@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 2047, 2048, 4100])
def test_prefixes_and_pages(vg, page, prefix):
    check(vg, 13, 4, 2, 4, 2, 64, torch.bfloat16, torch.bfloat16, page, prefix, [0, 3, 500, -7],
          heads_first=page == 48)


@pytest.mark.parametrize("prefix,B,hq,hkv,d", [(40000, 3, 2, 1, 128), (30011, 12, 2, 1, 256), (9000, 130, 16, 2, 64),
                                               (20011, 1, 1, 1, 64), (5003, 40, 5, 5, 128)])
@pytest.mark.parametrize("held", [None, E4M3])
def test_long_prefixes_cut_over_many_blocks(vg, prefix, B, hq, hkv, d, held):
    check(vg, 14, B, 1, hq, hkv, d, torch.bfloat16, held or torch.bfloat16, 64, prefix, [(11 * b) % 90 for b in range(B)])


def test_strided_q_scale_and_large_scores(vg):
    check(vg, 15, 3, 4, 6, 3, 96, torch.bfloat16, torch.bfloat16, 32, 300, [9, 40, 0], scale=0.3, strided=True)
    check(vg, 16, 3, 4, 6, 3, 128, torch.float16, torch.float16, 32, 300, [9, 40, 0], q_scale=60.0)
    check(vg, 17, 3, 4, 6, 3, 128, torch.bfloat16, torch.bfloat16, 32, 300, [9, 40, 0], scale=-0.1)
    check(vg, 18, 2, 20, 6, 3, 128, torch.bfloat16, torch.bfloat16, 32, 300, [9, 40], scale=0.0)


def test_nodes_that_see_no_draft(vg):
    tree = [[0, 0b10, 0b101, 0], [0, 0, 0b1, 0b1111], [-1, -1, -1, -1], [0, 0, 0, 0]]
    check(vg, 19, 4, 4, 4, 2, 64, torch.bfloat16, torch.bfloat16, 16, 70, [0, 33, 0, -70], tree=tree, counts=[4, 3, 0, 4],
          poison=True)


def test_missing_pages_of_the_prefix(vg):
    check(vg, 20, 3, 4, 4, 2, 64, torch.bfloat16, torch.bfloat16, 16, 100, [9, 60, 0], break_pages=True)
    check(vg, 21, 3, 4, 4, 2, 64, torch.bfloat16, torch.bfloat16, 16, 32, [0, 0, 0], break_pages=True)


def test_a_prefix_without_pages_and_one_past_its_pages(vg):
    """No pages: nothing is shared.  A length past the pages: they are all there is."""
    g = torch.Generator().manual_seed(22)
    q = randn(g, 2, 3, 4, 64, dtype=torch.bfloat16)
    cache, k, v, table, pages = build(vg, g, 2, 2, 64, 16, torch.bfloat16, torch.bfloat16, 64, [80, 90], 3, (1.0, 1.0))
    table[:, :4] = pages
    lens = torch.tensor([80, 90], dtype=torch.int32, device=DEV)
    want = vg.tree_attention(q, cache, lens)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    tp = torch.tensor([64], dtype=torch.int32, device=DEV)
    assert torch.equal(vg.prefix_attention(q, cache, lens, tp, none), want)
    for p in (64, 79, 2 ** 31 - 1, -5, 0):
        tp.fill_(p)
        got = vg.prefix_attention(q, cache, lens, tp, pages)
        # both are within (u + 2e) sum p |v| + u |o| of the formula's: |v| and e as above, sum p |v| below 1.5
        assert ((got.double() - want.double()).abs() <= 4 * (2.0 ** -8) * 1.5 + 2.0 ** -8 * want.double().abs()).all()


def test_one_workspace_for_calls_in_turn_and_other_prefixes(vg):
    g = torch.Generator().manual_seed(23)
    q = randn(g, 40, 4, 16, 128, dtype=torch.bfloat16)
    cache, *_ = build(vg, g, 40, 2, 128, 16, torch.bfloat16, torch.bfloat16, 0, [0] * 40, 4, (1.0, 1.0))
    ws = vg.prefix_attention_workspace(q, cache)
    check(vg, 24, 40, 4, 16, 2, 128, torch.bfloat16, torch.bfloat16, 64, 3000, [b for b in range(40)], workspace=ws)
    check(vg, 25, 3, 1, 4, 2, 128, torch.bfloat16, torch.bfloat16, 64, 9000, [5, 0, 900], workspace=ws)
    check(vg, 26, 40, 1, 16, 2, 128, torch.bfloat16, torch.bfloat16, 16, 100, [b for b in range(40)], workspace=ws)


def test_captured_calls_follow_the_device_words(vg):
    """Captured once, replayed at other prefixes and lengths; two graphs share a workspace."""
    g = torch.Generator().manual_seed(27)
    B, n, page = 3, 2, 16
    q = randn(g, B, n, 4, 64, dtype=torch.bfloat16)
    cache, k, v, table, pages = build(vg, g, B, 2, 64, page, torch.bfloat16, torch.bfloat16, 1600, [2000, 1700, 1900], n,
                                      (1.0, 1.0))
    table[:, :100] = pages
    lens = torch.tensor([2000, 1700, 1900], dtype=torch.int32, device=DEV)
    tp = torch.tensor([1600], dtype=torch.int32, device=DEV)
    ws = vg.prefix_attention_workspace(q, cache)
    side = torch.cuda.Stream()
    graphs = []
    for scale in (0.1, 0.2):
        vg.prefix_attention(q, cache, lens, tp, pages, scale=scale, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            graphs.append((graph, vg.prefix_attention(q, cache, lens, tp, pages, scale=scale, workspace=ws), scale))
    for prefix, now in ((1600, (2000, 1700, 1900)), (33, (100, 40, 1990)), (1000, (1000, 999, 0)), (0, (5, 6, 7))):
        tp.fill_(prefix)
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        for graph, out, scale in graphs:
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, vg.prefix_attention(q, cache, lens, tp, pages, scale=scale, workspace=ws))


def test_calls_on_two_streams_and_what_they_make(vg):
    """The output and the workspace that a call is not given are made on its stream."""
    g = torch.Generator().manual_seed(28)
    q = randn(g, 8, 4, 8, 128, dtype=torch.bfloat16)
    cache, k, v, table, pages = build(vg, g, 8, 2, 128, 64, torch.bfloat16, torch.bfloat16, 4096, [4200] * 8, 4, (1.0, 1.0))
    lens = torch.full((8,), 4200, dtype=torch.int32, device=DEV)
    tp = torch.tensor([4096], dtype=torch.int32, device=DEV)
    want = vg.prefix_attention(q, cache, lens, tp, pages)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(400_000_000)
    held = torch.cuda.Event()
    held.record()
    got = [vg.prefix_attention(q, cache, lens, tp, pages, stream=side) for _ in range(3)]
    side.synchronize()
    early = not held.query()
    both = [vg.prefix_attention(q, cache, lens, tp, pages, stream=s) for s in (side, torch.cuda.current_stream()) * 3]
    torch.cuda.synchronize()
    assert early
    assert all(torch.equal(x, want) for x in got + both)


def test_a_row_without_numbers_stays_without(vg):
    g = torch.Generator().manual_seed(29)
    cache, k, v, table, pages = build(vg, g, 3, 2, 64, 16, torch.bfloat16, torch.bfloat16, 256, [300, 260, 256], 3, (1.0, 1.0))
    q = randn(g, 3, 3, 4, 64, dtype=torch.bfloat16)
    lens = torch.tensor([300, 260, 256], dtype=torch.int32, device=DEV)
    tp = torch.tensor([256], dtype=torch.int32, device=DEV)
    want = vg.prefix_attention(q, cache, lens, tp, pages)
    q[1, 1, 0] = math.nan
    lse = torch.empty((3, 3, 4), device=DEV)
    got = vg.prefix_attention(q, cache, lens, tp, pages, lse=lse)
    assert torch.isnan(got[1, 1, 0]).all() and torch.isnan(lse[1, 1, 0])
    got[1, 1, 0], want[1, 1, 0] = 0, 0
    assert torch.equal(got, want)


def test_refusals(vg):
    g = torch.Generator().manual_seed(30)
    cache, k, v, table, pages = build(vg, g, 2, 2, 64, 16, torch.bfloat16, torch.bfloat16, 64, [80, 90], 3, (1.0, 1.0))
    q = randn(g, 2, 3, 4, 64, dtype=torch.bfloat16)
    lens = torch.tensor([80, 90], dtype=torch.int32, device=DEV)
    tp = torch.tensor([64], dtype=torch.int32, device=DEV)

    def call(q=q, lens=lens, prefix=tp, pages=pages, **kw):
        return vg.prefix_attention(q, cache, lens, prefix, pages, **kw)

    call()
    for kw in (dict(prefix=tp.long()), dict(prefix=tp[0]), dict(prefix=tp.cpu()), dict(prefix=None),
               dict(prefix=torch.zeros(2, dtype=torch.int32, device=DEV)), dict(pages=pages.long()), dict(pages=None),
               dict(pages=table), dict(pages=torch.zeros(8, dtype=torch.int32, device=DEV)[::2]), dict(pages=pages.cpu()),
               dict(q=q.half()), dict(q=q[:, :, :3]), dict(lens=lens[:1]), dict(scale=math.nan),
               dict(workspace=torch.zeros(64, dtype=torch.uint8, device=DEV)),
               dict(workspace=vg.tree_attention_workspace(q, cache)), dict(lse=torch.empty(3, device=DEV)),
               dict(q=randn(g, 2, 65, 4, 64, dtype=torch.bfloat16))):
        with pytest.raises((ValueError, vg.VGError)):
            call(**kw)
