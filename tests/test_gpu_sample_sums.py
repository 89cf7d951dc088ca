"""Draws from rows of which one logit is far above a long body of equal ones: what the body weighs together counts,
however little each of it does.

Here everything has a closed form: with a body of weight w = e^(-d / T) each and the large one at index t, the running sum
up to index i is (i + 1) w, and 1 - w more from t on.

Tolerance.  A weight is good to 2^-27.6 of itself (the table 2^-30, the series' last rounding 2^-29, the rounding down to
2^-30 of an octave's top 2^-29) and is rounded down to 2^-56 of the largest; sums are exact.  So the sum of V <= 2^28 of them is
off by 2^-27.6 of itself and 2^-28 of the largest, which weighs less than the sum, and a boundary's and u's share of it by
less than EDGE = 2^-26 together.  Differences of logits here are
exact.  A probability is off by (|z| + 4) 2^-22 of itself (ex2 of a product; z in octaves), and by what the sum is.
"""
import math

import pytest
import torch
from test_gpu_sample import check
from test_gpu_verify_round import DEV, randn, vg  # noqa: F401

pytestmark = pytest.mark.gpu

EDGE = 2.0 ** -26


def row(V, at, d, dtype):
    x = torch.zeros((1, V), dtype=dtype, device=DEV)
    x[0, at] = d
    return x


def numbers(V, at, w):
    """Random numbers at both sides of the large logit, within the body before and behind it, at the ends."""
    S = 1 + (V - 1) * w
    u = [0.0, at * w / S / 2, at * w / S, (at * w + 1) / S, (at * w + 0.5) / S, 0.25, 0.5, 0.75, 1 - 2.0 ** -24]
    u += [1 - (V - at) * w / S * f for f in (0.9, 0.5, 0.1)] + [1 - 2.0 ** -e for e in (9, 12, 16, 20)]
    return torch.tensor([u], dtype=torch.float32).clamp(0, 1 - 2.0 ** -24).to(DEV)


def hold(tokens, u, V, at, w, kept, S):
    """`kept` tokens of the order weigh S; those of the body come by index."""
    last = kept - 2 if kept - 2 < at else kept - 1       # the largest index of the body that is kept
    for i, v in zip(tokens.cpu().tolist(), u.cpu().double().tolist()):
        assert 0 <= i <= max(last, at), (i, v)
        below = min(i, kept - 1) * w if i <= at else (i - 1) * w + 1
        above = below + (1 if i == at else w)
        assert below <= (v + EDGE) * S and above >= (v - EDGE) * S, (i, v, (below / S - v) * 2 ** 26, (v - above / S) * 2 ** 26)


# octaves that a body lies below the largest: what it weighs in all goes from all to nothing that counts
@pytest.mark.parametrize("octaves", [12.0, 17.3, 20.0, 23.9, 28.5, 31.3, 33.0, 34.99, 35.5, 41.2, 57.0])
@pytest.mark.parametrize("V,dtype", [(33, torch.float32), (151936, torch.bfloat16), (151936, torch.float32),
                                     (1 << 20, torch.float16), (2500001, torch.bfloat16), (2500001, torch.float32)])
def test_one_above_a_body(vg, V, dtype, octaves):
    at, d = V // 3, 24.0
    T = torch.tensor([d / (octaves * math.log(2))], dtype=torch.float32)
    z = d / float(T[0])
    w, T = math.exp(-z), T.to(DEV)
    x, u = row(V, at, d, dtype), numbers(V, at, w)
    S = 1 + (V - 1) * w
    out = torch.empty((1, V), device=DEV)
    tokens = vg.sample(x, u, T, out=out)
    hold(tokens[0], u[0], V, at, w, V, S)
    off = (z / math.log(2) + 4) * 2.0 ** -22
    body = (out[0, :at], out[0, at + 1:])
    assert all(((b.double() - w / S).abs() <= (off + 2 * EDGE) * w / S + 1e-40).all() for b in body)
    assert abs(float(out[0, at]) - 1 / S) <= (2.0 ** -20 + EDGE) / S
    assert abs(float(out.double().sum()) - 1) <= 2.0 ** -20 / S + off * (V - 1) * w / S + 2 * EDGE
    # cut within the body by top-p and by top-k, alone and both
    for p, k in ((1 - (V - 1) * w / S / 2, 0), (1.0, V // 2), ((1 + (V // 2) * w / 4) / (1 + (V // 2) * w), V // 2 + 1)):
        p = float(torch.tensor(p, dtype=torch.float32).clamp(max=1 - 2.0 ** -24)) if p < 1 else 1.0
        first = k if 0 < k < V else V
        of = 1 + (first - 1) * w
        need = lambda t: max(1, min(first, 1 + math.ceil((t - 1) / w)))                   # noqa: E731
        least, most = (need((p + e) * of) if p < 1 else first for e in (-EDGE, EDGE))
        tokens = vg.sample(x, u, T, torch.tensor([k], dtype=torch.int32, device=DEV), torch.tensor([p], device=DEV), out=out)
        kept = int((out > 0).sum()) if w > 1e-30 else least
        assert least <= kept <= most, (p, k, least, kept, most)
        assert bool(out[0, at] > 0) and bool((out[0, :kept - 1 if kept - 1 <= at else kept] > 0).all())
        hold(tokens[0], u[0], V, at, w, kept, 1 + (kept - 1) * w)


@pytest.mark.parametrize("octaves", [27.0, 35.5, 38.25])
def test_the_longest_vocabularies(vg, octaves):
    """2^27 tokens and the most there may be."""
    d = 24.0
    for V, dtype in ((1 << 27, torch.float32), ((1 << 28) - 1, torch.bfloat16)):
        at = 12345
        T = torch.tensor([d / (octaves * math.log(2))], dtype=torch.float32)
        w, T = math.exp(-d / float(T[0])), T.to(DEV)
        x, u = row(V, at, d, dtype), numbers(V, at, w)
        S = 1 + (V - 1) * w
        hold(vg.sample(x, u, T)[0], u[0], V, at, w, V, S)
        p = float(torch.tensor(1 - (V - 1) * w / S / 2, dtype=torch.float32))
        need = lambda t: 1 + math.ceil((t - 1) / w)                                        # noqa: E731
        least, most = need((p - EDGE) * S), need((p + EDGE) * S)
        tokens = vg.sample(x, u, T, top_p=torch.tensor([p], device=DEV))[0]
        # the last of them all that is kept: drawn by the largest u there is, to 2^-24 of the sum
        i, room = int(tokens[8]), (2.0 ** -24 + EDGE) * S / w
        assert i > at and least - 1 - room <= i <= most - 1, (i, least, most, room)
        del x


@pytest.mark.parametrize("dtype,V", [(torch.float32, 1000003), (torch.bfloat16, 151936), (torch.float16, 700001)])
def test_one_above_many_of_all_sizes(vg, dtype, V):
    """A body that spreads over some twenty octaves, most of it far below the largest."""
    g = torch.Generator().manual_seed(31)
    x = randn(g, 2, V, dtype=dtype, scale=2.0) - 20
    x[0, 77], x[1, V - 9] = 0.0, 1.0
    u = torch.cat((torch.rand((2, 4), generator=g), 1 - 2.0 ** -torch.arange(3, 15).float().expand(2, 12)), 1).to(DEV)
    check(vg, x, u)
    check(vg, x, u, T=[1.0, 1.2], k=[0, V // 2], p=[0.9999, 0.9995])
