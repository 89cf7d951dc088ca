"""Whole rounds of a batch behind a shared prefix: norms and rotation with the append,
attention, draws from truncated distributions and their verification, one after
another over one cache, eagerly and captured."""
import pytest
import torch
from test_gpu_prefix_attention import build
from test_gpu_verify_round import DEV, randn, u, vg  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("held", [None, torch.float8_e4m3fn])
def test_rounds_behind_a_prefix(vg, held):
    g = torch.Generator().manual_seed(1)
    B, n, hq, hkv, d, V, page, prefix = 5, 4, 8, 2, 64, 5003, 16, 300
    dt = torch.bfloat16
    scales = (0.05, 0.05) if held else (1.0, 1.0)
    start = [300, 301, 317, 350, 288]                    # behind the prefix, and one in its last page
    cache, ck, cv, table, pages = build(vg, g, B, hkv, d, page, dt, held or dt, prefix, [s + 60 for s in start], n, scales)
    # a second cache over the same memory whose table names the shared pages, too
    full = table.clone()
    full[:, :len(pages)] = pages
    whole = vg.KVCache(ck, cv, full, *scales)
    wq, wk = 1 + randn(g, d, scale=0.2), 1 + randn(g, d, scale=0.2)
    inv, factor = vg.rope_frequencies(d, base=1e6, device=DEV)
    head = randn(g, hq * d, V, scale=0.2)
    lens = torch.tensor(start, dtype=torch.int32, device=DEV)
    tp = torch.tensor([prefix], dtype=torch.int32, device=DEV)
    temperature = torch.tensor([0.7, 0.0, 1.2, 1.0, 0.9], device=DEV).repeat_interleave(n)
    top_k = torch.tensor([40, 0, 0, 900, 5], dtype=torch.int32, device=DEV).repeat_interleave(n)
    top_p = torch.tensor([0.95, 0.9, 0.8, 1.0, 0.5], device=DEV).repeat_interleave(n)
    parents = torch.arange(-1, n - 1, dtype=torch.int32, device=DEV).expand(B, n).contiguous()
    q, k, v = (torch.empty((B, n, h, d), dtype=dt, device=DEV) for h in (hq, hkv, hkv))
    rnd, rnd2, noise = torch.empty((B, n), device=DEV), torch.empty((B, n), device=DEV), torch.empty((B * n, V), device=DEV)
    p, dq = torch.empty((B * n, V), device=DEV), torch.empty((B * n, V), device=DEV)
    ws = vg.prefix_attention_workspace(q, cache)

    def step():
        qr = vg.qk_norm_rope_append(q, k, v, wq, wk, inv, cache, lens, factor=factor)
        o = vg.prefix_attention(qr, cache, lens, tp, pages, workspace=ws)
        logits = o.float().view(B * n, hq * d) @ head
        args = dict(temperature=temperature, top_k=top_k, top_p=top_p)
        # drafts: node i's token is drawn from a rougher row after node i - 1
        drawn = vg.sample(logits + noise, rnd2.view(-1), out=dq, **args).view(B, n)
        tokens = torch.roll(drawn, 1, 1).contiguous()
        vg.sample(logits, rnd.view(-1), out=p, **args)
        accepted, path, out = vg.verify_tree(p.view(B, n, V), dq.view(B, n, V), tokens, parents, rnd)
        return qr, o, tokens, accepted, out

    def fresh():
        for t, s in ((q, 1.0), (k, 1.0), (v, 1.0), (noise, 0.2)):
            t.copy_(randn(g, *t.shape, dtype=t.dtype, scale=s))
        rnd.copy_(torch.rand((B, n), generator=g))
        rnd2.copy_(torch.rand((B, n), generator=g))

    fresh()
    step()
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        captured = step()
    some = 0
    for _ in range(6):
        fresh()
        eager = [t.clone() for t in step()]
        qr, o, tokens, accepted, out = eager
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager))
        # attention: as over the whole table, each within (u + 2e) sum p |v| + u |o| of the formula's,
        # sum p |v| below 2 for normal v and e below u here
        want = vg.tree_attention(qr, whole, lens)
        assert ((o.double() - want.double()).abs() <= 2 * (3 * u(dt) * 2 + u(dt) * want.double().abs())).all()
        a, t, pp = accepted.tolist(), out.tolist(), p.view(B, n, V)
        for b in range(B):
            some += a[b]
            assert t[b][:a[b]] == tokens[b, 1:a[b] + 1].tolist() and t[b][a[b] + 1:] == [-1] * (n - a[b])
            for i in range(a[b] + 1):                    # every token is one that the target keeps
                assert pp[b, i, t[b][i]] > 0
        lens += accepted + 1
    assert some > 0 and vg.workspace_error(ws) == 0
