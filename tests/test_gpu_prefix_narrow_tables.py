"""Attention behind a prefix of more pages than a sequence's row of the table has: the prefix's slots are named by its own pages, so
a sequence that is long enough has all of them, whatever its row could hold.  Tolerances: test_gpu_prefix_attention's."""
import math

import pytest
import torch
from test_gpu_verify_round import DEV, E4M3, randn, reference_attention, u, vg  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,held", [(torch.bfloat16, None), (torch.float16, None), (torch.bfloat16, E4M3)])
@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 2), (128, 40, 1), (256, 6, 2)])
@pytest.mark.parametrize("whole,columns", [(5, 1), (5, 4), (40, 3), (3, 3)])
def test_rows_of_the_table_shorter_than_the_prefix(vg, dtype, held, d, hq, hkv, whole, columns):
    g = torch.Generator().manual_seed(whole + columns)
    page, n, group = 16, 3, hq // hkv
    held, scales = held or dtype, (0.03, 0.05) if held else (1.0, 1.0)
    shared, room = whole * page, columns * page
    # all of the prefix and nothing more, more, shorter than it, as long as the row, nothing
    lens = [shared, shared + 3, shared + 500, shared - 1, room, 7, 0]
    B = len(lens)
    total = whole + B * columns
    order = torch.randperm(total, generator=g).to(torch.int32)
    pages, table = order[:whole].to(DEV), order[whole:].reshape(B, columns).to(DEV)
    k, v = (randn(g, total, page, hkv, d, scale=1 / s).to(held) for s in scales)
    cache = vg.KVCache(k, v, table, *scales)
    q = randn(g, B, n, hq, d, dtype=dtype)
    lse = torch.empty((B, n, hq), device=DEV)
    out = vg.prefix_attention(q, cache, torch.tensor(lens, dtype=torch.int32, device=DEV),
                              torch.tensor([shared + 5], dtype=torch.int32, device=DEV), pages, lse=lse)
    for b in range(B):
        path = (pages.tolist() if lens[b] >= shared else []) + table[b].tolist()[whole if lens[b] >= shared else 0:]
        slots = [s for s in range(lens[b] + n) if s // page < len(path)]
        at = torch.tensor([path[s // page] for s in slots], device=DEV), torch.tensor([s % page for s in slots], device=DEV)
        seen = torch.tensor([[s <= lens[b] + i for s in slots] for i in range(n)], device=DEV)
        for h in range(hkv):
            kk, vv = (t[at[0], at[1], h].double() * c for t, c in ((k, scales[0]), (v, scales[1])))
            rows = q[b, :, h * group:(h + 1) * group].double().reshape(n * group, d)
            see = seen[:, None, :].expand(n, group, len(slots)).reshape(n * group, len(slots))
            o, ls, a, e, av = reference_attention(rows, kk, vv, see, d ** -0.5)
            y = out[b, :, h * group:(h + 1) * group].double().reshape(n * group, d)
            l2 = lse[b, :, h * group:(h + 1) * group].double().reshape(-1)
            assert see.any(-1).all()
            tol = (u(dtype) + 2 * e) * a + u(dtype) * o.abs() + 1e-7 + (2.0 ** -25 * av if dtype == torch.float16 else 0)
            assert ((y - o).abs() <= tol).all(), (b, h)
            assert ((l2 - ls).abs() <= e[:, 0] + 2.0 ** -20 * (1 + ls.abs())).all(), (b, h)
            assert not math.isnan(float(l2.sum()))
