"""Cases of the operators of a verify round: rotary positions with the append
to a paged cache, attention of a tree of drafted tokens over that cache, the
probabilities of a row of logits, and the verification of the drafted tokens.

A tree's node 0 is the last committed token and nodes 1..n-1 are drafted;
node i of sequence b lies in the cache at slot lens[b] + i and its position
is lens[b] + depth[b, i].  Where ``own`` is false ``run`` computes the plain
form in elementary torch operations; where it is true it makes the calls of
verify_gemm_gb300.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # Decode without drafts, one request: the q, k and v of one 5120-wide
        # layer (40 heads of 128).  Latency is all there is.
        rope("rope, one token", B=1, n=1, hq=40, hkv=40, d=128, rot=128, layout="half", dtype="bf16",
             cache="same", page=64, past=4001, scaling="none", tree=False),
        # A batch's verify step far into long contexts: trees of 8 nodes, half
        # of the head rotated in interleaved pairs, an 8-bit cache.
        rope("rope, batch of trees", B=32, n=8, hq=40, hkv=8, d=128, rot=64, layout="interleaved",
             dtype="bf16", cache="e4m3", page=16, past=200000, scaling="yarn", tree=True),
        # A prompt taken into the cache in one go: bandwidth counts.
        rope("rope, prompt", B=1, n=16381, hq=40, hkv=8, d=128, rot=128, layout="half", dtype="fp16",
             cache="same", page=64, past=0, scaling="yarn", tree=False),
        # The first tokens of a chat with a small model.
        attention("attend, one short token", B=1, n=1, hq=32, hkv=8, d=64, dtype="bf16", cache="same",
                  page=16, length=130, tree=False),
        # The verify pass of the 64-layer stack: 8 columns, 40 heads of 128,
        # each with keys of its own.
        attention("attend, chain of 8", B=1, n=8, hq=40, hkv=40, d=128, dtype="bf16", cache="same", page=64,
                  length=8003, tree=False),
        # One request near the end of a 262144-token context, 8-bit cache.
        attention("attend, long context", B=1, n=4, hq=40, hkv=8, d=128, dtype="bf16", cache="e4m3", page=64,
                  length=262001, tree=False),
        # A serving batch of ragged lengths with trees of 16 nodes.
        attention("attend, ragged batch", B=48, n=16, hq=32, hkv=8, d=128, dtype="fp16", cache="same", page=16,
                  length=6007, tree=True),
        # The widest trees over shared heads: 512 rows read each key, so the
        # products and not the cache set the pace.
        attention("attend, wide trees", B=8, n=64, hq=64, hkv=8, d=128, dtype="bf16", cache="same", page=128,
                  length=8190, tree=True),
        # The head's row of one decode step.
        probabilities("probabilities, one row", rows=1, vocab=151936, dtype="bf16", temperature="one"),
        # Every node of a batch of chains, each request with a temperature of
        # its own, some of them greedy.
        probabilities("probabilities, batch", rows=256, vocab=151936, dtype="bf16", temperature="rows"),
        # One request's chain of 7 drafts.
        verify("verify, chain of 7", B=1, n=8, vocab=151936, tree=False),
        # A batch of trees with siblings that are tried one after another.
        verify("verify, batch of trees", B=48, n=16, vocab=151936, tree=True),
    ]


def rope(name, **c):
    return {"name": name, "op": "rope", **c}


def attention(name, **c):
    return {"name": name, "op": "attention", **c}


def probabilities(name, **c):
    return {"name": name, "op": "probabilities", **c}


def verify(name, **c):
    return {"name": name, "op": "verify", **c}


def log_int(rng, low, high):
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5))))))


def draw(rng):
    op = rng.choice(["rope", "attention", "attention", "attention", "probabilities", "verify"])
    if op in ("rope", "attention"):
        hkv, group = rng.choice([1, 2, 4, 5, 8, 16, 40]), rng.choice([1, 1, 2, 4, 5, 8])
        if hkv == 40:
            group = 1
        c = {"op": op, "hq": hkv * group, "hkv": hkv, "d": rng.choice([64, 80, 96, 128, 128, 128, 192, 256]),
             "dtype": rng.choice(["bf16", "fp16"]), "cache": rng.choice(["same", "same", "e4m3"]),
             "page": rng.choice([16, 32, 48, 64, 128])}
    if op == "rope":
        n = rng.choice([log_int(rng, 1, 64), log_int(rng, 64, 16384)])
        width = n * (c["hq"] + 2 * c["hkv"]) * c["d"]
        most = max(1, min(256, 16381 * 56 * 128 // width))
        if width > 16381 * 56 * 128:
            n = 16381 * 56 * 128 // ((c["hq"] + 2 * c["hkv"]) * c["d"])
        c.update(B=log_int(rng, 1, most), n=n, rot=rng.choice([c["d"], c["d"], c["d"] // 2, 16]),
                 layout=rng.choice(["half", "interleaved"]), past=rng.choice([0, log_int(rng, 1, 500000)]),
                 scaling=rng.choice(["none", "yarn"]), tree=n <= 64 and rng.random() < 0.5)
        return c
    if op == "attention":
        n = log_int(rng, 1, 64)
        B = log_int(rng, 1, 64)
        per_key = B * c["hkv"] * c["d"] * 4
        per_key_flops = 4 * B * c["hq"] * n * c["d"]
        most = min(150000, 500_000_000 // per_key, 120_000_000_000 // per_key_flops)
        c.update(B=B, n=n, length=log_int(rng, 1, most), tree=rng.random() < 0.5)
        return c
    if op == "probabilities":
        vocab = rng.choice([rng.randrange(1000, 32000), rng.randrange(32000, 200000), 151936])
        return {"op": op, "rows": log_int(rng, 1, min(512, 256 * 151936 // vocab)), "vocab": vocab,
                "dtype": rng.choice(["bf16", "fp16", "fp32"]), "temperature": rng.choice(["one", "rows"])}
    vocab = rng.choice([rng.randrange(1000, 32000), rng.randrange(32000, 200000), 151936])
    n = log_int(rng, 2, 32)
    return {"op": op, "B": log_int(rng, 1, min(128, 48 * 16 * 151936 // (n * vocab))), "n": n, "vocab": vocab,
            "tree": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs

def lengths(c, gen):
    """Committed tokens per sequence: one sequence has the whole length, the
    others' fall evenly to a fifth of it; which one is which goes by the seed."""
    top = c["length"]
    each = torch.tensor([top - (top * 4 * b) // (5 * c["B"]) for b in range(c["B"])], dtype=torch.int32)
    return each[torch.randperm(c["B"], generator=gen)]


def some_trees(B, n, gen):
    """parents, depths, ancestor words and node counts of random trees."""
    parents = torch.full((B, n), -1, dtype=torch.int32)
    depth = torch.zeros((B, n), dtype=torch.int32)
    words = [[1] for _ in range(B)]
    lean = torch.rand((B, n), generator=gen)
    for b in range(B):
        for i in range(1, n):
            at = max(0, i - 1 - int(float(lean[b, i]) ** 2 * min(i, 4)))
            parents[b, i] = at
            depth[b, i] = depth[b, at] + 1
            words[b].append(words[b][at] | (1 << i))
    signed = [[w - (1 << 64) if w >= 1 << 63 else w for w in row] for row in words]
    counts = torch.randint(max(1, n - n // 4), n + 1, (B,), generator=gen, dtype=torch.int32)
    return parents, depth, torch.tensor(signed, dtype=torch.int64), counts


def frequencies(rot, scaling):
    """(inverse frequencies in 64 bits, attention factor): base 1e6, and for
    "yarn" a context of 32768 stretched 8 times: fast pairs as they are, slow
    ones divided by 8, a ramp between."""
    j = torch.arange(rot // 2, dtype=torch.float64)
    inv = 1e6 ** (-2.0 * j / rot)
    if scaling == "none":
        return inv, 1.0
    turns = 32768 * inv / (2 * math.pi)
    keep = ((torch.log(turns) - math.log(1.0)) / (math.log(32.0) - math.log(1.0))).clamp(0, 1)
    return inv * keep + inv / 8 * (1 - keep), 0.1 * math.log(8) + 1.0


def paged(c, slots_first, slots_end, gen, device):
    """A shuffled page table that has pages for slots [first, end) of each
    sequence, and how many pages there are (a page for every sequence more
    than the slots need at least); other entries name page 0."""
    B, page = c["B"], c["page"]
    first, last = slots_first // page, (slots_end + page - 1) // page
    held = last - first
    start = torch.cumsum(held, 0) - held
    total = B + sum((int(k) + page - 1) // page for k in slots_end - slots_first)
    order = torch.randperm(total, generator=gen, dtype=torch.int64).to(torch.int32)
    col = torch.arange(int(last.max()))[None, :]
    inside = (col >= first[:, None]) & (col < last[:, None])
    index = torch.where(inside, start[:, None] + col - first[:, None], 0)
    return torch.where(inside, order[index], 0).to(torch.int32).to(device), total


def prepare(case, seed):
    c = dict(case)
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(scale)

    if c["op"] in ("rope", "attention"):
        dt = TYPES[c["dtype"]]
        held = E4M3 if c["cache"] == "e4m3" else dt
        B, n, hq, hkv, d = c["B"], c["n"], c["hq"], c["hkv"], c["d"]
        s["k_scale"], s["v_scale"] = (0.015, 0.02) if held == E4M3 else (1.0, 1.0)
        counts = None
        if c["tree"]:
            _, depth, words, counts = some_trees(B, n, host)
            s["depth"], s["words"] = depth.cuda(), words.cuda()
        s["counts"] = counts.cuda() if counts is not None else None
    if c["op"] == "rope":
        # what a projection wrote: q, k and v beside each other
        qkv = normal(B, n, hq + 2 * hkv, d, dtype=dt)
        s["q"], s["k"], s["v"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
        past = torch.full((B,), c["past"], dtype=torch.int64)
        if c["past"]:
            past -= torch.randint(0, 1 + c["past"] // 2, (B,), generator=host)
        # only the pages that this step writes: nothing else is touched
        s["table"], pages = paged(c, past, past + n, host, "cuda")
        s["lens"] = past.to(torch.int32).cuda()
        inv, s["factor"] = frequencies(c["rot"], c["scaling"])
        s["inv_freq"] = inv.cuda()
        s["ck"] = torch.zeros((pages, c["page"], hkv, d), dtype=held, device="cuda")
        s["cv"] = torch.zeros((pages, c["page"], hkv, d), dtype=held, device="cuda")
    elif c["op"] == "attention":
        lens = lengths(c, host)
        s["lens"] = lens.cuda()
        s["q"] = normal(B, n, hq, d, dtype=dt)
        s["table"], pages = paged(c, torch.zeros(B, dtype=torch.int64), lens.long() + n, host, "cuda")
        for key, scale in (("ck", s["k_scale"]), ("cv", s["v_scale"])):
            if held == E4M3:
                at = torch.empty((pages, c["page"], hkv, d), dtype=E4M3, device="cuda")
                for p0 in range(0, pages, 4096):
                    at[p0:p0 + 4096] = normal(min(4096, pages - p0), c["page"], hkv, d, scale=1 / scale).to(E4M3)
            else:
                at = normal(pages, c["page"], hkv, d, dtype=dt)
            s[key] = at
    elif c["op"] == "probabilities":
        s["x"] = normal(c["rows"], c["vocab"], scale=2.5, dtype=TYPES[c["dtype"]])
        s["temperature"] = None
        if c["temperature"] == "rows":
            t = 0.5 + torch.rand(c["rows"], generator=host)
            t[torch.rand(c["rows"], generator=host) < 0.1] = 0.0
            s["temperature"] = t.cuda()
    else:
        B, n, V = c["B"], c["n"], c["vocab"]
        rows = n if c["tree"] else n - 1
        # a draft that agrees with the target more often than not
        p = normal(B, n, V, scale=2.5)
        q = normal(B, rows, V, scale=0.6).add_(p[:, :rows])
        s["p"] = torch.softmax(p, -1)
        s["q"] = torch.softmax(q, -1)
        if c["tree"]:
            parents, _, _, counts = some_trees(B, n, host)
            s["counts"] = counts.cuda()
        else:
            parents, s["counts"] = torch.arange(-1, n - 1, dtype=torch.int32).expand(B, n).contiguous(), None
        s["parents"] = parents.cuda()
        # drafted tokens come from q of the parent: the largest of log q + Gumbel noise
        tokens = torch.full((B, n), -1, dtype=torch.int32, device="cuda")
        batch = torch.arange(B, device="cuda")
        for i in range(1, n):
            noise = torch.rand((B, V), generator=gen, device="cuda").clamp_(1e-12).log_().neg_().log_().neg_()
            tokens[:, i] = (noise + q[batch, s["parents"][:, i].long()]).argmax(-1).to(torch.int32)
        s["tokens"] = tokens
        s["u"] = torch.rand((B, n), generator=gen, device="cuda")
    if own:
        import verify_gemm_gb300 as vg

        if c["op"] in ("rope", "attention"):
            s["cache"] = vg.KVCache(s["ck"], s["cv"], s["table"], s["k_scale"], s["v_scale"])
        if c["op"] == "attention":
            s["workspace"] = vg.tree_attention_workspace(s["q"], s["cache"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    if c["op"] == "rope":
        return run_rope(c, s)
    if c["op"] == "attention":
        return run_attention(c, s)
    if c["op"] == "probabilities":
        return run_probabilities(s)
    return run_verify(c, s)


def of_cache(t):
    """8-bit codes as the values they stand for (before the scale): exact in bf16."""
    return t.to(torch.bfloat16) if t.dtype == E4M3 else t


def run_rope(c, s):
    depth = s["depth"] if c["tree"] else None
    if own:
        import verify_gemm_gb300 as vg

        q = vg.rope_append(s["q"], s["k"], s["v"], s["inv_freq"], s["cache"], s["lens"], depth=depth,
                           counts=s["counts"], layout=c["layout"], factor=s["factor"])
        return q, of_cache(s["ck"]), of_cache(s["cv"])
    B, n, rot = c["B"], c["n"], c["rot"]
    steps = torch.arange(n, device="cuda")
    at = s["lens"].double()[:, None] + (depth if depth is not None else steps[None, :]).double()
    angle = at[:, :, None] * s["inv_freq"]
    cos, sin = ((f(angle) * s["factor"]).float()[:, :, None, :] for f in (torch.cos, torch.sin))

    def turned(x):
        x = x.float()
        if c["layout"] == "half":
            x1, x2 = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat((x1 * cos - x2 * sin, x1 * sin + x2 * cos), -1)
        else:
            x1, x2 = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack((x1 * cos - x2 * sin, x1 * sin + x2 * cos), -1).flatten(-2)
        return torch.cat((y, x[..., rot:]), -1)

    def held(x, scale, dtype):
        return (x / scale).clamp(-448, 448).to(dtype) if dtype == E4M3 else x.to(dtype)

    used = steps[None, :] < (s["counts"][:, None] if s["counts"] is not None else n)
    slot = s["lens"].long()[:, None] + steps
    page = torch.gather(s["table"].long(), 1, slot // c["page"])
    if s["counts"] is None:
        index = (page, slot % c["page"])
        s["ck"][index] = held(turned(s["k"]), s["k_scale"], s["ck"].dtype)
        s["cv"][index] = held(s["v"].float(), s["v_scale"], s["cv"].dtype)
        return turned(s["q"]).to(s["q"].dtype), of_cache(s["ck"]), of_cache(s["cv"])
    index = (page[used], (slot % c["page"])[used])
    # written as bytes: 8-bit floats have no masked store of their own
    for cache, x, scale in ((s["ck"], turned(s["k"]), s["k_scale"]), (s["cv"], s["v"].float(), s["v_scale"])):
        whole = torch.int8 if cache.dtype == E4M3 else torch.int16
        cache.view(whole)[index] = held(x[used], scale, cache.dtype).view(whole)
    q = torch.where(used[:, :, None, None], turned(s["q"]), 0.0).to(s["q"].dtype)
    return q, of_cache(s["ck"]), of_cache(s["cv"])


def run_attention(c, s):
    B, n, hq, hkv, d = c["B"], c["n"], c["hq"], c["hkv"], c["d"]
    words = s["words"] if c["tree"] else None
    if own:
        import verify_gemm_gb300 as vg

        lse = torch.empty((B, n, hq), dtype=torch.float32, device="cuda")
        out = vg.tree_attention(s["q"], s["cache"], s["lens"], tree=words, counts=s["counts"], lse=lse,
                                workspace=s["workspace"])
        return out, lse
    page = c["page"]
    slots = s["table"].shape[1] * page
    steps = torch.arange(n, device="cuda")
    counts = s["counts"] if s["counts"] is not None else torch.full_like(s["lens"], n)

    def dense(cache, scale):  # [B, hkv, slots, d]
        return cache[s["table"].long()].float().mul_(scale).reshape(B, slots, hkv, d).transpose(1, 2)

    q = s["q"].float().reshape(B, n, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, -1, d)
    score = torch.matmul(q, dense(s["ck"], s["k_scale"]).transpose(2, 3)).mul_(d ** -0.5)
    key = torch.arange(slots, device="cuda")
    draft = key[None, :] - s["lens"][:, None]                                   # [B, slots]
    if words is None:
        seen = draft[:, None, :] <= steps[None, :, None]
    else:
        seen = (words[:, :, None] >> draft.clamp(0, 63)[:, None, :]) & 1 == 1
    seen = torch.where(draft[:, None, :] < 0, True, seen) & (draft < counts[:, None])[:, None, :]
    seen = seen & (steps[None, :] < counts[:, None])[:, :, None]                # [B, n, slots]
    seen = seen[:, None, :, None, :].expand(B, 1, n, hq // hkv, slots).reshape(B, 1, -1, slots)
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score.sub_(torch.where(top == -math.inf, 0.0, top)))
    total = p.sum(-1, keepdim=True)
    held = (key[None, :] < (s["lens"] + counts)[:, None])[:, None, :, None]
    o = torch.matmul(p, torch.where(held, dense(s["cv"], s["v_scale"]), 0.0)) / torch.where(total == 0, 1.0, total)
    lse = torch.log(total) + torch.where(top == -math.inf, 0.0, top)

    def rows(x):
        return x.reshape(B, hkv, n, hq // hkv, -1).permute(0, 2, 1, 3, 4).reshape(B, n, hq, -1)

    return rows(o).to(s["q"].dtype), rows(lse)[..., 0]


def run_probabilities(s):
    if own:
        import verify_gemm_gb300 as vg

        return vg.probabilities(s["x"], temperature=s["temperature"])
    x = s["x"].float()
    top = x.amax(-1, keepdim=True)
    if s["temperature"] is None:
        e = torch.exp(x - top)
        return e / e.sum(-1, keepdim=True)
    t = s["temperature"][:, None]
    greedy = t <= 0
    e = torch.exp((x - top) / torch.where(greedy, 1.0, t))
    e = e / e.sum(-1, keepdim=True)
    token = torch.arange(x.shape[-1], device="cuda")
    first = torch.where(x == top, token, x.shape[-1]).amin(-1, keepdim=True)
    return torch.where(greedy, (token == first).float(), e)


def run_verify(c, s):
    if own:
        import verify_gemm_gb300 as vg

        return vg.verify_tree(s["p"], s["q"], s["tokens"], s["parents"], s["u"], counts=s["counts"])
    p, q, tokens, u, n, rows = s["p"], s["q"], s["tokens"].long(), s["u"].double(), c["n"], s["q"].shape[1]
    batch = torch.arange(c["B"], device="cuda")
    counts = s["counts"] if s["counts"] is not None else torch.full_like(batch, n)
    cur, accepted = torch.zeros_like(batch), torch.zeros_like(batch)
    a, total = torch.zeros_like(u[:, 0]), torch.ones_like(u[:, 0])
    path = torch.full((c["B"], n), -1, dtype=torch.int32, device="cuda")
    out = torch.full((c["B"], n + 1), -1, dtype=torch.int32, device="cuda")
    places = torch.arange(n + 1, device="cuda")

    def residual(cur, a):
        drafted = q[batch, cur.clamp(max=rows - 1)].double()
        return (p[batch, cur].double() - a[:, None] * drafted).clamp(min=0)

    for i in range(1, n):
        tried = (s["parents"][:, i] == cur) & (i < counts)
        token = tokens[:, i].clamp(min=0)
        qt = q[batch, cur.clamp(max=rows - 1), token].double()
        rt = (p[batch, cur, token].double() - a * qt).clamp(min=0)
        taken = tried & (u[:, i] * qt * total < rt)
        refused = tried & ~taken
        here = taken[:, None] & (places[None, :] == accepted[:, None])
        path = torch.where(here[:, :n], i, path)
        out = torch.where(here, tokens[:, i, None].to(torch.int32), out)
        accepted = accepted + taken.long()
        cur = torch.where(taken, i, cur)
        a = torch.where(taken, 0.0, torch.where(refused, a + total, a))
        total = torch.where(taken, 1.0, torch.where(refused, residual(cur, a).sum(-1), total))
    left = residual(cur, a)
    left = torch.where(left.sum(-1, keepdim=True) > 0, left, p[batch, cur].double())
    sums = left.cumsum(-1)
    last = torch.searchsorted(sums, (u[:, 0] * sums[:, -1])[:, None], right=True)[:, 0].clamp(max=c["vocab"] - 1)
    out = torch.where(places[None, :] == accepted[:, None], last[:, None].to(torch.int32), out)
    return accepted.to(torch.int32), path, out


# ---------------------------------------------------------------- what it takes

def work(case):
    c = case
    if c["op"] == "rope":
        tokens = c["B"] * c["n"]
        size = 2
        held = 1 if c["cache"] == "e4m3" else 2
        return {"bytes": tokens * c["d"] * (2 * size * c["hq"] + (size + held) * 2 * c["hkv"]),
                "flops": tokens * 3 * c["rot"] * (c["hq"] + c["hkv"])}
    if c["op"] == "attention":
        held = 1 if c["cache"] == "e4m3" else 2
        keys = sum(c["length"] - (c["length"] * 4 * b) // (5 * c["B"]) + c["n"] for b in range(c["B"]))
        rows = c["B"] * c["n"] * c["hq"]
        return {"bytes": 2 * keys * c["hkv"] * c["d"] * held + rows * (4 * c["d"] + 4),
                "flops": 4 * keys * c["hq"] * c["n"] * c["d"]}
    if c["op"] == "probabilities":
        size = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": c["rows"] * c["vocab"] * (size + 4), "flops": 3 * c["rows"] * c["vocab"]}
    # the row of the node where a sequence ends, and the draft's row there
    return {"bytes": c["B"] * (8 * c["vocab"] + 28 * c["n"]), "flops": 4 * c["B"] * c["vocab"]}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    if c["op"] == "rope":
        return exact_rope(c, s)
    if c["op"] == "attention":
        return exact_attention(c, s)
    if c["op"] == "probabilities":
        x = s["x"].double()
        t = s["temperature"].double() if s["temperature"] is not None else torch.ones(c["rows"], device="cuda").double()
        rows = []
        for r in range(c["rows"]):
            if float(t[r]) > 0:
                y = x[r] / t[r]
                rows.append(torch.exp(y - torch.logsumexp(y, 0)))
            else:
                y = torch.zeros_like(x[r])
                y[int((x[r] == x[r].max()).nonzero()[0])] = 1.0
                rows.append(y)
        return torch.stack(rows)
    return exact_verify(c, s)


def exact_rope(c, s):
    """The rotation as a product of complex numbers, token by token where the trees differ."""
    B, n, rot = c["B"], c["n"], c["rot"]
    depth = s["depth"] if c["tree"] else torch.arange(n, device="cuda").expand(B, n)
    position = (s["lens"].long()[:, None] + depth.long()).double()
    turn = torch.polar(torch.full((B, n, 1, rot // 2), s["factor"], dtype=torch.float64, device="cuda"),
                       (position[:, :, None] * s["inv_freq"])[:, :, None, :])

    def turned(x):
        x = x.double().clone()
        pairs = (slice(0, rot // 2), slice(rot // 2, rot)) if c["layout"] == "half" else (slice(0, rot, 2), slice(1, rot, 2))
        z = torch.complex(x[..., pairs[0]], x[..., pairs[1]]) * turn
        x[..., pairs[0]], x[..., pairs[1]] = z.real, z.imag
        return x

    counts = s["counts"].tolist() if s["counts"] is not None else [n] * B
    lens, table, page = s["lens"].tolist(), s["table"].long(), c["page"]
    q, k, v = turned(s["q"]), turned(s["k"]) / s["k_scale"], s["v"].double() / s["v_scale"]
    ck, cv = (torch.zeros(s[key].shape, dtype=torch.float64, device="cuda") for key in ("ck", "cv"))
    for b in range(B):
        q[b, counts[b]:] = 0
        slot = torch.arange(lens[b], lens[b] + counts[b], device="cuda")
        at = table[b, slot // page], slot % page
        ck[at], cv[at] = k[b, :counts[b]], v[b, :counts[b]]
    if c["cache"] == "e4m3":  # the code is a choice between neighbours: a value that it stands for has no 64-bit form
        return q, None, None
    return q, ck, cv


def exact_attention(c, s):
    B, n, hq, hkv, d = c["B"], c["n"], c["hq"], c["hkv"], c["d"]
    out = torch.zeros((B, n, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, n, hq), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        length = int(s["lens"][b])
        count = int(s["counts"][b]) if s["counts"] is not None else n
        slot = torch.arange(length + count, device="cuda")
        at = s["table"][b].long()[slot // c["page"]], slot % c["page"]
        see = torch.ones((count, length + count), dtype=torch.bool, device="cuda")
        if c["tree"]:
            bits = [[(int(w) >> j) & 1 for j in range(count)] for w in s["words"][b, :count].tolist()]
            see[:, length:] = torch.tensor(bits, device="cuda").bool()
        else:
            see[:, length:] = torch.ones((count, count), device="cuda").tril().bool()
        for g in range(hkv):
            k = s["ck"][at[0], at[1], g].double() * s["k_scale"]
            v = s["cv"][at[0], at[1], g].double() * s["v_scale"]
            heads = slice(g * (hq // hkv), (g + 1) * (hq // hkv))
            x = torch.einsum("ihd,jd->hij", s["q"][b, :count, heads].double(), k) / math.sqrt(d)
            x = torch.where(see[None], x, -math.inf)
            norm = torch.logsumexp(x, -1)
            out[b, :count, heads] = torch.einsum("hij,jd->ihd", torch.exp(x - norm[..., None]), v)
            lse[b, :count, heads] = norm.T
    return out, lse


def exact_verify(c, s):
    """Sequence by sequence, with the residual kept as a distribution and renewed at each refusal."""
    accepted, path, out = [], [], []
    for b in range(c["B"]):
        count = int(s["counts"][b]) if s["counts"] is not None else c["n"]
        parents, tokens, u = s["parents"][b].tolist(), s["tokens"][b].tolist(), s["u"][b].double().tolist()
        nodes, cur = [], 0
        r, weight = s["p"][b, 0].double(), 1.0
        for i in range(1, count):
            if parents[i] != cur:
                continue
            q = s["q"][b, cur].double()
            if u[i] * float(q[tokens[i]]) * weight < float(r[tokens[i]]):
                nodes.append(i)
                cur, r, weight = i, s["p"][b, i].double(), 1.0
            else:
                r = torch.relu(r - weight * q)
                weight = float(r.sum())
        if float(r.sum()) <= 0:
            r = s["p"][b, cur].double()
        sums = torch.cumsum(r, 0)
        last = min(int((sums <= u[0] * sums[-1]).sum()), c["vocab"] - 1)
        accepted.append(len(nodes))
        path.append(nodes + [-1] * (c["n"] - len(nodes)))
        out.append([tokens[i] for i in nodes] + [last] + [-1] * (c["n"] - len(nodes)))
    return tuple(torch.tensor(x, dtype=torch.int32) for x in (accepted, path, out))
