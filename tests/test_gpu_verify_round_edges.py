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
