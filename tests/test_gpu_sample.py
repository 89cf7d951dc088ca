"""Draws from truncated distributions, against 64 bits.

Tolerances.  A weight is exact to 2^-28 of itself (the table's and the series' 2^-30
each, the rounding to units of 2^-29; 16-bit logits below 2^-16 of the largest:
2^-24 z, for z of at most some 40 octaves 2^-18, of tokens that weigh 2^-z), and sums
are exact, so which token a draw or a limit of weight ends on is only open where
the formula's sums lie within EDGE = 2^-26 of the whole from it.  A probability
goes by ex2 of a product: |z| 2^-23 from the product and the difference, 2^-22
from ex2 and 2^-22 from the division and its factors, so it is off by less than (|z| + 4) 2^-22.
"""
import math

import pytest
import torch
from test_gpu_verify_round import DEV, randn, vg  # noqa: F401

pytestmark = pytest.mark.gpu

EDGE = 2.0 ** -26
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def reference(x, T, k, p, mp):
    """(kept tokens in order, how many may be kept: least and most, weights in order, z) of one row in 64 bits."""
    x = x.double().cpu()
    V = len(x)
    if torch.isnan(x).any() or math.isnan(T) or (T > 0 and x.max() == math.inf) or x.max() == -math.inf:
        return None
    order = torch.sort(x, descending=True, stable=True).indices
    if T <= 0:
        return order, 1, 1, torch.ones(V, dtype=torch.float64), torch.zeros(V, dtype=torch.float64)
    z = (x[order[0]] - x[order]) / T
    z = torch.where(x[order] == -math.inf, math.inf, z)
    w = torch.exp(-z)
    most = int((x > -math.inf).sum())
    if 0 < k < V:
        most = min(most, k)
    least = most
    if p < 1:
        sums = torch.cumsum(w[:most], 0)
        want = p * float(sums[-1])
        edge = EDGE * float(sums[-1])
        first = lambda t: int((sums < t).sum()) + 1                      # noqa: E731
        least, most = (max(1, min(most, first(t))) for t in (want - edge, want + edge))
    if mp > 0:
        n = max(1, int((w >= mp).sum()))
        least, most = min(least, n), min(most, n)
    return order, least, most, w, z / math.log(2)


def check(vg, x, u, T=None, k=None, p=None, mp=None):
    """One call on rows x [R, V] with draws u [R, D]; the settings are lists or None."""
    R, V = x.shape
    f = lambda v, t: None if v is None else torch.tensor(v, dtype=t, device=DEV)         # noqa: E731
    args = dict(temperature=f(T, torch.float32), top_k=f(k, torch.int32), top_p=f(p, torch.float32),
                min_p=f(mp, torch.float32))
    out = torch.full((R, V), 7.0, device=DEV)
    got = vg.sample(x, u, out=out, **args)
    assert got.dtype == torch.int32 and got.shape == u.shape
    assert torch.equal(got, vg.sample(x, u, **args))
    out, tokens, uu = out.cpu().double(), got.cpu().reshape(R, -1), u.cpu().double().reshape(R, -1)
    one = lambda v, r, default: default if v is None else float(torch.tensor(v[r], dtype=torch.float32))  # noqa: E731
    for r in range(R):
        t = one(T, r, 1.0)
        ref = reference(x[r], t, 0 if k is None else k[r], one(p, r, 1.0), one(mp, r, 0.0))
        if ref is None:
            assert (tokens[r] == -1).all()
            none = t <= 0 or not (torch.isnan(x[r].float()).any() or x[r].float().max() == math.inf or math.isnan(t))
            assert (out[r] == 0).all() if none else torch.isnan(out[r]).all()
            continue
        order, least, most, w, z = ref
        # what is kept is a beginning of the order, as long as it may be
        n = int((out[r][order] > 0).sum())
        tiny = int((w[:most] < 2.0 ** -120).sum())                       # weights that FP32 may not hold
        assert least - tiny <= n <= most and (out[r][order[n:]] == 0).all(), (r, n, least, most)
        keep = order[:max(n, min(least, most))]
        sum_w = float(w[:len(keep)].sum())
        want = w[:n] / sum_w
        assert ((out[r][order[:n]] - want).abs() <= (z[:n] + 4) * 2.0 ** -22 * want + 1e-37).all(), r
        at = torch.sort(keep)
        sums = torch.cumsum(w[:len(keep)][at.indices], 0)
        for d in range(tokens.shape[1]):
            v = float(uu[r, d])
            v = 0.0 if not v > 0 else min(v, 1 - 2.0 ** -24)
            i = int(tokens[r, d])
            j = int(torch.searchsorted(at.values, i))
            assert j < len(keep) and at.values[j] == i, (r, d, i)        # a token that is kept
            below = float(sums[j - 1]) if j else 0.0
            assert below <= (v + EDGE) * sum_w and float(sums[j]) >= (v - EDGE) * sum_w, (r, d)
            assert w[:len(keep)][at.indices[j]] > 0


def settings(g, R, V):
    T = [float(t) for t in 0.3 + 1.5 * torch.rand(R, generator=g)]
    k = [int(v) for v in torch.randint(0, max(2, min(V, 400)), (R,), generator=g)]
    p = [float(v) for v in torch.rand(R, generator=g) * 1.1]
    mp = [float(v) for v in torch.rand(R, generator=g) ** 6]
    for r in range(R):
        if r % 5 == 1:
            k[r] = 0
        if r % 4 == 2:
            p[r] = 1.0
        if r % 3:
            mp[r] = 0.0
        if r % 7 == 6:
            T[r] = 0.0
    return T, k, p, mp


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (5, 7), (9, 33), (21, 1000), (400, 1500), (11, 4097), (7, 2049),
                                        (9, 50257), (3, 151936), (70, 151936), (1, 200003)])
def test_rows_and_vocabularies(vg, dtype, rows, vocab):
    g = torch.Generator().manual_seed(rows + vocab)
    x = randn(g, rows, vocab, dtype=dtype, scale=2.5)
    u = torch.rand((rows, 3), generator=g).to(DEV)
    if rows > 50:                                        # the reference sorts each row here
        check(vg, x[:24].contiguous(), u[:24].contiguous(), *[s[:24] for s in settings(g, rows, vocab)])
        T, k, p, mp = settings(g, rows, vocab)
        t = lambda v, d: torch.tensor(v, dtype=d, device=DEV)            # noqa: E731
        args = (t(T, torch.float32), t(k, torch.int32), t(p, torch.float32), t(mp, torch.float32))
        out = torch.empty((rows, vocab), device=DEV)
        all_rows = vg.sample(x, u, *args, out=out)
        for r in (0, 25, rows - 1):                      # a row alone gives what it gives among others
            alone = torch.empty((1, vocab), device=DEV)
            assert torch.equal(vg.sample(x[r:r + 1], u[r:r + 1], *[a[r:r + 1] for a in args], out=alone)[0], all_rows[r])
            assert torch.equal(alone[0], out[r])
        return
    check(vg, x, u, *settings(g, rows, vocab))
    check(vg, x, u)


@pytest.mark.parametrize("dtype,vocab", [(torch.bfloat16, 20000), (torch.float32, 9001)])
@pytest.mark.parametrize("rows", [305, 511, 512, 513])
@pytest.mark.parametrize("which", ["all", "slow rows last", "none slow", "all slow", "top-k alone", "top-p alone"])
def test_rows_begin_in_any_order(vg, dtype, vocab, rows, which):
    """Many rows, of which those that take longest may begin first: each is what it is among few."""
    g = torch.Generator().manual_seed(rows)
    x = randn(g, rows, vocab, dtype=dtype, scale=2.5)
    u = torch.rand((rows, 2), generator=g).to(DEV)
    T, k, p, mp = settings(g, rows, vocab)
    if which != "all":
        k, p = [40] * rows, [1.0] * rows
    if which in ("slow rows last", "all slow"):
        n = 3 if which == "slow rows last" else rows
        k[rows - n:], p[rows - n:], T[rows - n:] = [0] * n, [0.8] * n, [0.9] * n
    t = lambda v, d: torch.tensor(v, dtype=d, device=DEV)                # noqa: E731
    args = dict(temperature=t(T, torch.float32), top_k=t(k, torch.int32), top_p=t(p, torch.float32),
                min_p=t(mp, torch.float32))
    if which.endswith("alone"):
        name = which.replace("-", "_").split()[0]
        args = {name: t([(250 if r % 3 else 30) if name == "top_k" else 0.2 + r % 5 / 5 for r in range(rows)],
                        torch.int32 if name == "top_k" else torch.float32)}
    out = torch.full((rows, vocab), 7.0, device=DEV)
    tokens = vg.sample(x, u, out=out, **args)
    assert torch.equal(tokens, vg.sample(x, u, **args))
    for at in range(0, rows, 61):
        few = torch.empty_like(out[at:at + 61])
        part = vg.sample(x[at:at + 61], u[at:at + 61], out=few, **{n: a[at:at + 61] for n, a in args.items()})
        assert torch.equal(part, tokens[at:at + 61]) and torch.equal(few, out[at:at + 61]), at
    check(vg, x[-4:], u[-4:], *[None if n not in args else args[n][-4:].tolist()
                                for n in ("temperature", "top_k", "top_p", "min_p")])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("k", [0, -3, 1, 2, 50, 199, 200, 201, 1000, 4999, 5000, 5001, 2 ** 31 - 1])
def test_top_k(vg, dtype, k):
    g = torch.Generator().manual_seed(k % 1000)
    x = randn(g, 3, 5000, dtype=dtype, scale=2.0)
    x[1] = (x[1] * 2).round() / 2                        # many equal logits
    u = torch.rand((3, 4), generator=g).to(DEV)
    check(vg, x, u, k=[k] * 3)
    check(vg, x, u, T=[0.7] * 3, k=[k] * 3, p=[0.6, 0.6, 0.999], mp=[0.0, 0.01, 0.1])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("p", [-1.0, 0.0, 1e-30, 1e-7, 0.3, 0.9, 0.999999, 1 - 2.0 ** -24, 1.0, 7.0])
def test_top_p(vg, dtype, p):
    g = torch.Generator().manual_seed(5)
    x = randn(g, 4, 30011, dtype=dtype, scale=2.0)
    x[1] = (x[1] * 4).round() / 4
    x[2] += 100.0 * (torch.arange(30011, device=DEV) == 12345)           # one token has it all
    u = torch.rand((4, 2), generator=g).to(DEV)
    check(vg, x, u, p=[p] * 4)
    check(vg, x, u, T=[0.2, 3.0, 1.0, 30.0], p=[p] * 4)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("mp", [-1.0, 0.0, 1e-38, 1e-10, 0.05, 0.5, 1.0, 1.5])
def test_min_p(vg, dtype, mp):
    g = torch.Generator().manual_seed(6)
    x = randn(g, 3, 9001, dtype=dtype, scale=2.0)
    x[1] = (x[1] * 2).round() / 2
    u = torch.rand((3, 2), generator=g).to(DEV)
    check(vg, x, u, mp=[mp] * 3)
    check(vg, x, u, T=[0.5, 2.0, 0.0], p=[0.9] * 3, mp=[mp] * 3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 30])
@pytest.mark.parametrize("loud", [100, 129, 190, 300, 700, 1100, 2500])
def test_large_logits_in_one_place(vg, dtype, rows, loud):
    """A small top-k whose tokens all lie with one of a row's blocks, the first, one between or the last."""
    g = torch.Generator().manual_seed(loud)
    V = 151936
    x = randn(g, rows, V, dtype=dtype, scale=1.0)
    for r in range(rows):
        at = [0, 70001, V - loud][(r + loud) % 3]
        x[r, at:at + loud] += 20
    u = torch.rand((rows, 3), generator=g).to(DEV)
    n = min(rows, 3)
    check(vg, x[:n], u[:n], k=[200, 199, 50][:n], p=[0.9, 1.0, 0.99][:n])
    args = [torch.tensor(v, device=DEV) for v in ([1.0] * rows, [200, 199, 50] * 10, [0.9, 1.0, 0.99] * 10)]
    args = [args[0], args[1][:rows].to(torch.int32), args[2][:rows]]
    out = torch.empty((rows, V), device=DEV)
    got = vg.sample(x, u, args[0], top_k=args[1], top_p=args[2], out=out)
    for r in range(0, rows, 7):                          # (alone: on more blocks)
        alone = torch.empty((1, V), device=DEV)
        part = vg.sample(x[r:r + 1], u[r:r + 1], args[0][:1], top_k=args[1][r:r + 1], top_p=args[2][r:r + 1], out=alone)
        assert torch.equal(part[0], got[r]) and torch.equal(alone[0], out[r])


@pytest.mark.parametrize("dtype", TYPES)
def test_equal_logits(vg, dtype):
    """Rows of one value, of two, in order and against it: the lowest index goes first."""
    V = 20011
    i = torch.arange(V, device=DEV)
    x = torch.stack([torch.full((V,), -3.0, device=DEV), (i % 2).float(), (i >= V - 5).float() * 4, i.float() / V,
                     -i.float() / V, torch.zeros(V, device=DEV) * (1 - 2 * (i % 2))]).to(dtype)
    assert torch.signbit(x[5].float()).any()             # 0 and -0 are equal
    u = torch.tensor([[0.0, 0.25, 0.75, 1 - 2.0 ** -24]] * 6, device=DEV)
    for k, p, mp in ((0, 1.0, 0.0), (3, 1.0, 0.0), (150, 0.5, 0.0), (700, 1.0, 0.9), (0, 0.5, 0.0), (0, 0.001, 1.0),
                     (19999, 0.7, 0.0), (2500, 0.999, 0.5)):
        check(vg, x, u, T=[1.0, 0.5, 2.0, 1.0, 1.0, 3.0], k=[k] * 6, p=[p] * 6, mp=[mp] * 6)


@pytest.mark.parametrize("dtype,vocab", [(torch.bfloat16, 151936), (torch.float16, 700001), (torch.float32, 600007),
                                         (torch.float32, 1000003), (torch.bfloat16, 2500001)])
def test_long_rows(vg, dtype, vocab):
    """Rows that fill the shared memory of 16 blocks, and more; likely tokens beside each other."""
    g = torch.Generator().manual_seed(13)
    x = randn(g, 3, vocab, dtype=dtype, scale=2.0)
    x[1] = torch.sort(x[1].float(), descending=True).values.to(dtype)
    x[2, 1000:3000] += 6.0
    u = torch.rand((3, 2), generator=g).to(DEV)
    for T, k, p, mp in ((1.0, 0, 1.0, 0.0), (0.8, 60, 0.9, 0.0), (0.9, 200, 1.0, 0.001), (1.0, 0, 0.7, 0.0),
                        (1.1, 3000, 0.8, 0.0), (0.7, 0, 1.0, 0.2), (0.0, 0, 1.0, 0.0)):
        check(vg, x, u, T=[T] * 3, k=[k] * 3, p=[p] * 3, mp=[mp] * 3)


@pytest.mark.parametrize("dtype", TYPES)
def test_masked_rows(vg, dtype):
    """-infinity, the type's lowest value, infinities and NaN."""
    g = torch.Generator().manual_seed(7)
    V, low = 8003, torch.finfo(dtype).min
    x = randn(g, 12, V, dtype=dtype, scale=2.0)
    x[0, ::2] = -math.inf
    x[1, 1:] = -math.inf
    x[2] = -math.inf
    x[3, ::3] = low
    x[4] = low
    x[5, 77] = math.nan
    x[6, 5] = math.inf
    x[7, 5], x[7, 9] = math.inf, math.nan
    x[8, :-1] = -math.inf
    x[9, 100:] = low
    x[10] = torch.finfo(dtype).max
    x[11, :7999] = -math.inf
    u = torch.rand((12, 2), generator=g).to(DEV)
    for T, k, p, mp in ((1.0, 0, 1.0, 0.0), (0.7, 40, 0.9, 0.02), (0.0, 0, 1.0, 0.0), (1.3, 4500, 0.95, 0.0),
                        (1.0, 1, 1.0, 0.0), (1.0, 300, 1.0, 0.3)):
        check(vg, x, u, T=[T] * 12, k=[k] * 12, p=[p] * 12, mp=[mp] * 12)


@pytest.mark.parametrize("dtype", TYPES)
def test_temperatures(vg, dtype):
    """The ends of T: greedy at and below 0, one token for the smallest, all alike for the largest."""
    g = torch.Generator().manual_seed(8)
    T = [0.0, -0.0, -5.0, -math.inf, math.nan, 1e-45, 1e-38, 1e-6, 1e3, 1e36, 3e38, math.inf]
    x = randn(g, len(T), 3001, dtype=dtype, scale=3.0)
    u = torch.rand((len(T), 3), generator=g).to(DEV)
    check(vg, x, u, T=T)
    check(vg, x, u, T=T, k=[20] * len(T), p=[0.8] * len(T))
    check(vg, x, u, T=T, p=[0.8] * len(T), mp=[0.1] * len(T))


def test_random_numbers_at_their_ends(vg):
    g = torch.Generator().manual_seed(9)
    x = randn(g, 2, 5003, dtype=torch.float32)
    u = torch.tensor([[0.0, -0.0, 1e-45, 0.5, 1 - 2.0 ** -24, 1.0, 2.0, -1.0, math.nan, math.inf]] * 2, device=DEV)
    check(vg, x, u)
    check(vg, x, u, k=[30, 0], p=[1.0, 0.5])


@pytest.mark.parametrize("dtype", TYPES)
def test_logits_that_lie_apart(vg, dtype):
    """The first columns of a wider product; one row without a batch; many draws of a row."""
    g = torch.Generator().manual_seed(10)
    wide = randn(g, 6, 5120, dtype=dtype, scale=2.0)
    wide[:, 5001:] = math.inf                            # beside the rows: not theirs
    x, u = wide[:, :5001], torch.rand((6, 1), generator=g).to(DEV)
    check(vg, x, u, *settings(g, 6, 5001))
    check(vg, wide[:, :4999][1:5:3], u[:2].contiguous(), *settings(g, 2, 4999))
    y = x[2].contiguous()
    many = torch.rand(5000, generator=g).to(DEV)
    got = vg.sample(y, many, top_k=torch.tensor([700], dtype=torch.int32, device=DEV))
    assert got.shape == (5000,)
    check(vg, x[2:3].contiguous(), many[None], k=[700])
    # rows and distributions that begin between 16-byte borders
    flat = randn(g, 3 * 701 + 9, dtype=dtype, scale=2.0)
    room = torch.full((3 * 701 + 9,), 7.0, device=DEV)
    for first in range(1, 9):
        z, out = flat[first:first + 3 * 701].view(3, 701), room[first:first + 3 * 701].view(3, 701)
        want = torch.empty((3, 701), device=DEV)
        assert torch.equal(vg.sample(z, u[:3], out=out), vg.sample(z.clone(), u[:3], out=want))
        assert torch.equal(out, want) and (room[:1] == 7).all() and (room[first + 3 * 701:] == 7).all()
    alone = vg.sample(y, many[0])
    assert alone.shape == () and int(alone) == int(vg.sample(x[2:3], many[:1])[0])


def test_draws_are_distributed_as_the_row(vg):
    """Evenly spaced random numbers: each token comes up as often as its probability says, to one."""
    g = torch.Generator().manual_seed(11)
    x, n = randn(g, 1, 300, dtype=torch.float32, scale=1.5), 60000
    out = torch.empty_like(x)
    u = ((torch.arange(n) + 0.5) / n)[None].to(DEV)
    got = vg.sample(x, u, top_p=torch.tensor([0.9], device=DEV), out=out)
    counts = torch.bincount(got[0].long(), minlength=300)
    assert ((counts - out[0] * n).abs() <= 1 + n * 1e-5).all()


def test_captured_and_on_other_streams(vg):
    g = torch.Generator().manual_seed(12)
    x, u = randn(g, 5, 60001, dtype=torch.bfloat16, scale=2.0), torch.rand((5,), generator=g).to(DEV)
    T, k = torch.full((5,), 0.8, device=DEV), torch.tensor([0, 7, 300, 1, 0], dtype=torch.int32, device=DEV)
    p = torch.tensor([0.9, 0.5, 0.9, 1.0, 1.0], device=DEV)
    out = torch.empty((5, 60001), device=DEV)
    want = vg.sample(x, u, T, k, p, out=out).clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        got = vg.sample(x, u, T, k, p, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    x.copy_(randn(g, 5, 60001, dtype=torch.bfloat16))
    k.copy_(torch.tensor([9, 0, 0, 900, 2], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, vg.sample(x, u, T, k, p))
    torch.cuda._sleep(400_000_000)
    held = torch.cuda.Event()
    held.record()
    apart = vg.sample(x, u, T, k, p, stream=side)
    side.synchronize()
    early = not held.query()
    torch.cuda.synchronize()
    assert early and torch.equal(apart, got)


def test_refusals(vg):
    x, u = torch.zeros((2, 8), device=DEV), torch.zeros(2, device=DEV)
    vg.sample(x, u)
    for bad in (lambda: vg.sample(x.double(), u), lambda: vg.sample(x.cpu(), u), lambda: vg.sample(x, u.cpu()),
                lambda: vg.sample(x.t(), u), lambda: vg.sample(x[:, ::2], u), lambda: vg.sample(x[:0], u[:0]),
                lambda: vg.sample(x[:, :0], u), lambda: vg.sample(x[None], u), lambda: vg.sample(x, u[:1]),
                lambda: vg.sample(x, u.double()), lambda: vg.sample(x, u[0]), lambda: vg.sample(x, torch.zeros((2, 0), device=DEV)),
                lambda: vg.sample(x, torch.zeros((2, 2, 2), device=DEV)), lambda: vg.sample(x, torch.zeros((3, 2), device=DEV).t()),
                lambda: vg.sample(x[:1].expand(2, 8), u),
                lambda: vg.sample(x, u, temperature=torch.ones(3, device=DEV)),
                lambda: vg.sample(x, u, temperature=torch.ones(2, device=DEV).double()),
                lambda: vg.sample(x, u, top_k=torch.ones(2, dtype=torch.int64, device=DEV)),
                lambda: vg.sample(x, u, top_p=torch.ones(1, device=DEV)), lambda: vg.sample(x, u, min_p=0.1),
                lambda: vg.sample(x, u, out=torch.empty((2, 9), device=DEV)),
                lambda: vg.sample(x, u, out=torch.empty((2, 8), device=DEV).half())):
        with pytest.raises((ValueError, vg.VGError)):
            bad()
