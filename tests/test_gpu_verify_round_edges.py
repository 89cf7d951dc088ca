"""Borders of the verify round's operators: many refusals, temperatures at the ends of FP32,
logits that are not numbers, workspaces whose error word is set, dimensions of one.

Whole numbers are equal.  Probabilities are held to the bound of test_gpu_verify_round.py:
(x - max) / T and the exponential are off by |x - max| / T 2^-22 + 2^-21 relative, the sum's
additions by 2^-24 times their depth, which 2^-17 covers.
"""
import ctypes
import math

import pytest
import torch

from test_gpu_verify_round import DEV, E4M3, build_cache, randn, vg  # noqa: F401

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------- verification

# clusters of 2, 9, 2 and 8 blocks a sequence
@pytest.mark.parametrize("B,n,V", [(3, 64, 4099), (2, 300, 20000), (6, 1024, 4500), (16, 100, 40001)])
def test_verify_many_nodes_over_several_blocks(vg, B, n, V):
    """More nodes than a warp has lanes, rows that several blocks share out: against running
    sums in 64 bits.  Most children are refused, so that every node counts."""
    check_long(vg, *draw_long(11 + n, B, n, V), again=3)


def draw_long(seed, B, n, V):
    g = torch.Generator().manual_seed(seed)
    p = torch.softmax(torch.randn((B, n, V), generator=g) * 2.0, -1)
    rows = min(n, 12)
    q = torch.softmax(torch.randn((B, rows, V), generator=g) * 2.0, -1)
    parents = torch.full((B, n), -1, dtype=torch.int32)
    for b in range(B):
        for i in range(1, n):
            parents[b, i] = int(torch.randint(0, min(i, rows), (1,), generator=g))
    tokens = torch.full((B, n), -1, dtype=torch.int32)
    for b in range(B):
        for f in range(rows):
            mine = (parents[b] == f).nonzero()[:, 0]
            if len(mine):
                tokens[b, mine] = torch.multinomial(q[b, f], len(mine), replacement=True, generator=g).to(torch.int32)
    return p, q, tokens, parents, torch.rand((B, n), generator=g)


def check_long(vg, p, q, tokens, parents, u, again=1):
    B, n, V = p.shape
    p, q, tokens, parents, u = (t.to(DEV) for t in (p, q, tokens, parents, u))
    got = [vg.verify_tree(p, q, tokens, parents, u) for _ in range(again)]
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))
    acc, path, out = (t.tolist() for t in got[0])
    par, tok, uu = parents.tolist(), tokens.tolist(), u.double().tolist()
    for b in range(B):
        cur, r, S, kept = 0, p[b, 0].double(), 1.0, []
        for i in range(1, n):
            if par[b][i] != cur:
                continue
            t = tok[b][i]
            if uu[b][i] * float(q[b, cur, t]) * S < float(r[t]):
                kept.append(i)
                cur, r, S = i, p[b, i].double(), 1.0
                if cur >= q.shape[1]:
                    break
            else:
                r = (r - S * q[b, cur].double()).clamp(min=0)
                S = float(r.sum())
        if float(r.sum()) <= 0:
            r = p[b, cur].double()
        run = r.cumsum(0)
        last = int((run <= uu[b][0] * float(run[-1])).sum())
        assert acc[b] == len(kept) and path[b] == kept + [-1] * (n - len(kept)), b
        assert out[b] == [tok[b][i] for i in kept] + [last] + [-1] * (n - len(kept)), b


def test_verify_a_batch_over_a_real_vocabulary(vg):
    """Twelve sequences, eight blocks each."""
    check_long(vg, *draw_long(5, 12, 8, 151936))


def whole_verify(p, q, tokens, u, count):
    """The rule in whole numbers for children of the root alone: (accepted node or None, the last
    token).  p [nodes][V], q [V] and u [nodes] in units of 2^-24; the residual and its sum S in
    units of 2^-(24 + s)."""
    r, S, s, node = list(p[0]), 1 << 24, 0, None
    for i in range(1, count):
        if u[i] * q[tokens[i]] * S < r[tokens[i]] << 48:
            r, node = p[i], i
            break
        r = [max((a << 24) - S * b, 0) for a, b in zip(r, q)]
        S, s = sum(r), s + 24
    if sum(r) == 0:
        r = p[node or 0]
    run, last = 0, -1
    for k, x in enumerate(r):
        run += x
        if run << 24 > u[0] * sum(r):
            last = k
            break
    return node, last


def check_whole(vg, p, q, tokens, u, counts):
    """p [B, n, V], q [B, V], u [B, n] int64 in units of 2^-24, tokens [B, n]: all of the root's."""
    B, n, V = p.shape
    parents = torch.zeros((B, n), dtype=torch.int32)
    f = [(t.double() * 2.0 ** -24).float().to(DEV) for t in (p, q[:, None], u)]
    assert all(torch.equal((x.double() * 2 ** 24).long().cpu().view(t.shape), t) for x, t in zip(f, (p, q, u)))
    acc, path, out = vg.verify_tree(f[0], f[1], tokens.int().to(DEV), parents.to(DEV), f[2],
                                    counts=torch.tensor(counts, dtype=torch.int32, device=DEV))
    for b in range(B):
        node, last = whole_verify(p[b].tolist(), q[b].tolist(), tokens[b].tolist(), u[b].tolist(), counts[b])
        kept = [] if node is None else [node]
        assert path[b].tolist() == kept + [-1] * (n - len(kept)), b
        assert out[b].tolist() == [int(tokens[b, i]) for i in kept] + [last] + [-1] * (n - len(kept)), b
        assert int(acc[b]) == len(kept)


@pytest.mark.parametrize("V", [7, 8])
def test_verify_of_a_thousand_refusals(vg, V):
    """Nearly disjoint p and q: what q is weighed with passes 256 after some 350 refusals and
    reaches 600, while entries with a small q keep a residual."""
    g = torch.Generator().manual_seed(17)
    B, n, one = 10, 1024, 1 << 24
    p = torch.zeros((B, n, V), dtype=torch.long)
    p[:] = torch.tensor([0.3, 0.25, 0.2, 0.15, 0.1] + [0.0] * (V - 5)).mul(one).long()
    q = torch.zeros((B, V), dtype=torch.long)
    q[:, :5] = (torch.rand((B, 5), generator=g) * 0.002 * one).long()
    q[:, 0] = torch.linspace(0.0001, 0.0006, B).mul(one).long()
    q[:, V - 1] = one - q.sum(1)
    tokens = torch.full((B, n), V - 1)
    u = torch.randint(0, one, (B, n), generator=g)
    u[:, 0] = torch.linspace(0.01, 0.97, B).mul(one).long()
    counts = [1024, 350, 360, 400, 513, 700, 900, 1023, 1000, 600]
    for b in range(0, B, 2):
        tokens[b, counts[b] - 1] = b // 2 % 4            # the last child may hold
    check_whole(vg, p, q, tokens, u, counts)


def test_verify_of_rows_that_sum_to_nearly_sixteen(vg):
    g = torch.Generator().manual_seed(18)
    B, n, V, one = 8, 1000, 36, 1 << 24
    p = torch.zeros((B, n, V), dtype=torch.long)
    p[:, :, :16] = (0.99 * one * (1 - 0.01 * torch.rand((B, 1, 16), generator=g))).long()
    q = torch.zeros((B, V), dtype=torch.long)
    q[:, 18:34] = int(0.99 * one)
    q[:, :16] = (10.0 ** -torch.linspace(2, 4.5, 16) * one).long()
    tokens = torch.randint(18, 34, (B, n), generator=g)
    u = torch.randint(0, one, (B, n), generator=g)
    u[:, 0] = torch.linspace(0.01, 0.97, B).mul(one).long()
    counts = [5, 17, 18, 20, 40, 100, 500, 1000]
    for b in range(1, B, 2):
        tokens[b, counts[b] - 1] = 15
    check_whole(vg, p, q, tokens, u, counts)


# -------------------------------------------------------------- probabilities

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("vocab", [1, 8, 9, 1003, 4096, 20007, 151937])
def test_probabilities_at_the_ends_of_the_temperatures(vg, dtype, vocab):
    g = torch.Generator().manual_seed(vocab)
    temps = [math.inf, 3e38, 1e30, 1e-30, 5e-39, 1e-40, 1e-45, math.inf, 1e-40, math.inf, 1e-45]
    x = randn(g, len(temps), vocab, dtype=dtype, scale=2.5)
    x[7:9, 1::3] = -math.inf                             # masked by -infinity ...
    x[9:, 1::3] = torch.finfo(dtype).min                 # ... and by the lowest value
    t = torch.tensor(temps, dtype=torch.float32, device=DEV)
    xd = x.double()
    z = (xd - xd.amax(-1, keepdim=True)) / t.double()[:, None]
    z = torch.where(xd == -math.inf, -math.inf, z)       # (over an infinite T, too)
    want = torch.softmax(z, -1)
    tol = want * (z.abs().clamp(max=200) * 2.0 ** -22 + 2.0 ** -21 + 2.0 ** -17) + 1e-37
    got = vg.probabilities(x, temperature=t).double()
    assert ((got - want).abs() <= tol).all(), ((got - want).abs() - tol).amax(-1)


def test_probabilities_of_a_temperature_that_is_no_number(vg):
    x = randn(torch.Generator().manual_seed(2), 2, 1003)
    y = vg.probabilities(x, temperature=torch.tensor([math.nan, 1.0], device=DEV))
    assert torch.isnan(y[0]).all() and not torch.isnan(y[1]).any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,vocab", [(1, 5), (3, 1003), (40, 4099), (2, 151937), (4, 800011)])
def test_probabilities_of_greedy_rows_with_nan(vg, dtype, rows, vocab):
    """No logit is the largest beside a NaN: the row is 0, as a row without a logit is."""
    g = torch.Generator().manual_seed(rows)
    x = randn(g, rows, vocab, dtype=dtype)
    clean = vg.probabilities(x, temperature=torch.zeros(rows, device=DEV))
    assert (clean.sum(-1) == 1).all()
    for at in sorted({0, 1 % vocab, vocab // 2, vocab - 2, vocab - 1}):
        y = x.clone()
        row = at % rows
        y[row, at] = -math.nan if at % 2 else math.nan
        got = vg.probabilities(y, temperature=torch.zeros(rows, device=DEV))
        assert (got[row] == 0).all(), at
        sampled = vg.probabilities(y)
        assert torch.isnan(sampled[row]).all(), at
        keep = torch.arange(rows, device=DEV) != row
        assert torch.equal(got[keep], clean[keep]) and torch.isfinite(sampled[keep]).all()


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("n,hq,hkv,d,held", [
    (1, 8, 2, 64, None), (3, 10, 2, 64, None), (8, 4, 2, 128, None), (6, 4, 1, 128, E4M3), (20, 1, 1, 256, None),
    (20, 3, 1, 192, None), (64, 3, 1, 192, E4M3), (16, 8, 2, 128, None), (16, 8, 2, 64, E4M3),
    (64, 16, 2, 128, None), (64, 16, 2, 128, E4M3)])
def test_attention_of_a_workspace_whose_error_word_is_set(vg, n, hq, hkv, d, held):
    """Nothing that a call computes passes for a result before the error has been read and cleared."""
    g = torch.Generator().manual_seed(n)
    lens = [9000, 0, 30, 400]
    cache, *_ = build_cache(vg, g, 4, 9000 + n, hkv, d, 64, torch.bfloat16, held or torch.bfloat16,
                            (0.03, 0.04) if held else (1.0, 1.0))
    q = randn(g, 4, n, hq, d, dtype=torch.bfloat16)
    tl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    counts = torch.tensor([n, n, max(1, n - 1), n], dtype=torch.int32, device=DEV)
    ws = vg.tree_attention_workspace(q, cache)

    def call():
        lse = torch.zeros((4, n, hq), device=DEV)
        return vg.tree_attention(q, cache, tl, counts=counts, lse=lse, workspace=ws), lse

    want = call()
    ws[:4].view(torch.int32).fill_(16)
    used = (torch.arange(n, device=DEV)[None, :] < counts[:, None])
    for _ in range(2):
        out, lse = call()
        assert torch.isnan(out[used]).all() and torch.isnan(lse[used]).all()
        assert (out[~used] == 0).all() and (lse[~used] == -math.inf).all()
    assert vg.workspace_error(ws) == 16
    out, lse = call()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert vg.workspace_error(ws) == 0


def test_dimensions_of_one_may_have_any_stride(vg):
    """A single sequence, node or head, and a table of one column."""
    g = torch.Generator().manual_seed(4)
    d = 64
    for B, n, h in ((1, 3, 2), (2, 1, 2), (2, 3, 1), (1, 1, 1)):
        cache, *_ = build_cache(vg, g, B, 60, 1, d, 16, torch.bfloat16, torch.bfloat16)
        lens = torch.full((B,), 40, dtype=torch.int32, device=DEV)
        flat = randn(g, B * n * h * d, dtype=torch.bfloat16)
        q = flat.view(B, n, h, d)
        odd = torch.as_strided(flat, (B, n, h, d), [s if size > 1 else 7 for s, size in zip(q.stride(), q.shape)])
        assert torch.equal(odd, q)
        assert torch.equal(vg.tree_attention(odd, cache, lens), vg.tree_attention(q, cache, lens))
        kv = randn(g, B, n, 1, d, dtype=torch.bfloat16)
        inv, _ = vg.rope_frequencies(d, device=DEV)
        assert torch.equal(vg.rope_append(odd, kv, kv, inv, cache, lens), vg.rope_append(q, kv, kv, inv, cache, lens))
    k = randn(g, 4, 64, 1, d, dtype=torch.bfloat16)
    column = torch.as_strided(torch.tensor([2, 0], dtype=torch.int32, device=DEV), (2, 1), (1, 5))
    plain = column.contiguous().view(2, 1)
    q = randn(g, 2, 3, 1, d, dtype=torch.bfloat16)
    lens = torch.tensor([30, 11], dtype=torch.int32, device=DEV)
    assert torch.equal(vg.tree_attention(q, vg.KVCache(k, k, column), lens),
                       vg.tree_attention(q, vg.KVCache(k, k, plain), lens))


# ------------------------------------------------------- the cache's descriptor

def fake_cache(L, **kw):
    """A descriptor over addresses that nothing reads: it is only checked."""
    c = L.vg_kv_cache()
    c.k, c.v, c.page_table = 0x10000, 0x10000, 0x10000
    c.type, c.heads, c.head_dim, c.page_size, c.pages = L.VG_TYPE_E4M3, 2, 64, 16, 8
    for s in (c.k_stride, c.v_stride):
        s[0], s[1], s[2] = 16 * 128, 128, 64
    c.table_stride, c.batch, c.max_pages, c.k_scale, c.v_scale = 4, 3, 4, 0.5, 0.5
    for name, value in kw.items():
        setattr(c, name, value)
    return c


def test_a_cache_that_has_changed_is_refused(vg):
    from verify_gemm_gb300 import _lib as L

    n = ctypes.c_size_t()
    ask = lambda c: L.vg_tree_attention_workspace_size(4, 2, ctypes.byref(c), ctypes.byref(n))  # noqa: E731
    changes = dict(k=0x20000, v=0x20000, page_table=0x20000, type=L.VG_TYPE_BF16, heads=1, head_dim=32, page_size=32,
                   pages=9, table_stride=5, batch=2, max_pages=3, k_scale=0.25, v_scale=0.0)
    for name, value in changes.items():
        c = fake_cache(L)
        assert L.vg_kv_cache_init(ctypes.byref(c)) == 0 and ask(c) == 0
        setattr(c, name, value)
        assert ask(c) == 1, name
    for at in range(3):
        for name in ("k_stride", "v_stride"):
            c = fake_cache(L)
            assert L.vg_kv_cache_init(ctypes.byref(c)) == 0
            getattr(c, name)[at] += 64
            assert ask(c) == 1, (name, at)


def test_a_table_of_nearly_all_32_bit_slots_is_refused(vg):
    """A length and its tree's nodes have to fit 32 bits."""
    from verify_gemm_gb300 import _lib as L

    for slots, status in ((2 ** 31 - 16, 3), (2 ** 31 - 8192 + 16, 3), (2 ** 31 - 8192, 0)):
        c = fake_cache(L, max_pages=slots // 16, table_stride=slots // 16)
        assert L.vg_kv_cache_init(ctypes.byref(c)) == status, slots
