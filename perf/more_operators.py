"""Cases of more operators of a verify round: norms of the heads of q and k
with the rotary positions and the append in the same pass, tree attention of a
batch whose sequences share a long prefix, and sampling from truncated
distributions of logits.

The cache and the trees are those of the verify round: node i of sequence b
lies in the cache at slot lens[b] + i and its position is lens[b] +
depth[b, i].  Where ``own`` is false ``run`` computes the plain form in
elementary torch operations; where it is true it makes the calls of
verify_gemm_gb300.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # One token of one request through a layer of 40 heads of 128: latency.
        norms("norms, one token", B=1, n=1, hq=40, hkv=8, d=128, rot=128, layout="half", dtype="bf16",
              weights="bf16", cache="same", page=64, past=4001, scaling="none", tree=False),
        # A batch's verify step far into long contexts: trees of 8 nodes, half of
        # the head rotated in interleaved pairs, an 8-bit cache, FP32 weights.
        norms("norms, batch of trees", B=32, n=8, hq=40, hkv=8, d=128, rot=64, layout="interleaved", dtype="bf16",
              weights="fp32", cache="e4m3", page=16, past=200000, scaling="yarn", tree=True),
        # A prompt taken into the cache in one go: bandwidth counts.
        norms("norms, prompt", B=1, n=16381, hq=40, hkv=8, d=128, rot=128, layout="half", dtype="fp16",
              weights="fp16", cache="same", page=64, past=0, scaling="yarn", tree=False),
        # Two requests of a small model behind a short instruction.
        prefixed("prefix, two short requests", B=2, n=1, hq=32, hkv=8, d=64, dtype="bf16", cache="same", page=16,
                 prefix=500, own=130, tree=False),
        # Decode of a serving batch behind one system prompt.
        prefixed("prefix, decode of a batch", B=48, n=1, hq=40, hkv=8, d=128, dtype="bf16", cache="same", page=64,
                 prefix=8003, own=1201, tree=False),
        # Chains of 4 over a document that everybody asks about, 8-bit cache.
        prefixed("prefix, long document", B=16, n=4, hq=40, hkv=8, d=128, dtype="bf16", cache="e4m3", page=64,
                 prefix=65500, own=700, tree=False),
        # The verify pass of a large batch of trees: the products set the pace.
        prefixed("prefix, batch of trees", B=64, n=8, hq=64, hkv=8, d=128, dtype="fp16", cache="same", page=128,
                 prefix=16384, own=1000, tree=True),
        # The next token of one request.
        sampled("sample, one row", rows=1, draws=1, vocab=151936, dtype="bf16", filters="top-k 50, top-p 0.95",
                probs=False),
        # Four drafts of each of a few requests, independent draws from one row:
        # the verification needs the distribution that they were drawn from.
        sampled("sample, drafts", rows=8, draws=4, vocab=151936, dtype="bf16", filters="top-p 0.9", probs=True),
        # A serving batch of which each request has settings of its own.
        sampled("sample, mixed batch", rows=256, draws=1, vocab=151936, dtype="bf16", filters="mixed", probs=False),
        # The target's truncated distributions after each node of a batch's chains.
        sampled("sample, distributions", rows=128, draws=1, vocab=151936, dtype="fp32", filters="mixed", probs=True),
        # Temperature alone, a vocabulary of an odd size.
        sampled("sample, untruncated", rows=64, draws=1, vocab=32003, dtype="fp16", filters="none", probs=False),
    ]


def norms(name, **c):
    return {"name": name, "op": "norms", **c}


def prefixed(name, **c):
    return {"name": name, "op": "prefix", **c}


def sampled(name, **c):
    return {"name": name, "op": "sample", **c}


def log_int(rng, low, high):
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5))))))


def draw(rng):
    op = rng.choice(["norms", "prefix", "prefix", "sample", "sample"])
    if op == "sample":
        vocab = rng.choice([rng.randrange(1000, 32000), rng.randrange(32000, 200000), 151936])
        return {"op": op, "rows": log_int(rng, 1, min(512, 256 * 151936 // vocab)), "draws": rng.choice([1, 1, 2, 5]),
                "vocab": vocab, "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "filters": rng.choice(["none", "top-k 50, top-p 0.95", "top-p 0.9", "min-p 0.05", "mixed", "mixed"]),
                "probs": rng.random() < 0.5}
    hkv, group = rng.choice([1, 2, 4, 5, 8, 16, 40]), rng.choice([1, 1, 2, 4, 5, 8])
    if hkv == 40:
        group = 1
    c = {"op": op, "hq": hkv * group, "hkv": hkv, "d": rng.choice([64, 80, 96, 128, 128, 128, 192, 256]),
         "dtype": rng.choice(["bf16", "fp16"]), "cache": rng.choice(["same", "same", "e4m3"]),
         "page": rng.choice([16, 32, 48, 64, 128])}
    if op == "norms":
        n = rng.choice([log_int(rng, 1, 64), log_int(rng, 64, 16384)])
        width = (c["hq"] + 2 * c["hkv"]) * c["d"]
        n = min(n, 16381 * 56 * 128 // width)
        c.update(B=log_int(rng, 1, max(1, min(256, 16381 * 56 * 128 // (n * width)))), n=n,
                 rot=rng.choice([c["d"], c["d"], c["d"] // 2, 16]), layout=rng.choice(["half", "interleaved"]),
                 weights=rng.choice([c["dtype"], "fp32"]), past=rng.choice([0, log_int(rng, 1, 500000)]),
                 scaling=rng.choice(["none", "yarn"]), tree=n <= 64 and rng.random() < 0.5)
        return c
    n, B = log_int(rng, 1, 16), log_int(rng, 2, 128)
    rows = B * n * c["hq"]
    most = min(131072, 200_000_000 // (c["hkv"] * c["d"]), 130_000_000_000 // (4 * rows * c["d"]))
    prefix = log_int(rng, 64, max(64, most))
    own_most = min(2000, 200_000_000 // (B * c["hkv"] * c["d"]), 16_000_000_000 // (4 * rows * c["d"]))
    c.update(B=B, n=n, prefix=prefix, own=log_int(rng, 1, max(1, own_most)), tree=rng.random() < 0.5)
    return c


# ---------------------------------------------------------------- inputs

def some_trees(B, n, gen):
    """Depths, ancestor words and node counts of random trees."""
    depth = torch.zeros((B, n), dtype=torch.int32)
    words = [[1] for _ in range(B)]
    lean = torch.rand((B, n), generator=gen)
    for b in range(B):
        for i in range(1, n):
            at = max(0, i - 1 - int(float(lean[b, i]) ** 2 * min(i, 4)))
            depth[b, i] = depth[b, at] + 1
            words[b].append(words[b][at] | (1 << i))
    signed = [[w - (1 << 64) if w >= 1 << 63 else w for w in row] for row in words]
    counts = torch.randint(max(1, n - n // 4), n + 1, (B,), generator=gen, dtype=torch.int32)
    return depth, torch.tensor(signed, dtype=torch.int64), counts


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


def paged(page, slots_first, slots_end, shared, gen):
    """A page table with pages of a shuffled pool for slots [first, end) of each
    sequence, and the pool's size; `shared` pages of the pool, returned, too,
    are the first of every sequence.  Other entries name page 0."""
    first, last = slots_first // page, (slots_end + page - 1) // page
    held = last - first
    start = shared + torch.cumsum(held, 0) - held
    total = shared + len(held) + sum((int(k) + page - 1) // page for k in slots_end - slots_first)
    order = torch.randperm(total, generator=gen, dtype=torch.int64).to(torch.int32)
    col = torch.arange(max(1, int(last.max())))[None, :]
    inside = (col >= first[:, None]) & (col < last[:, None])
    index = torch.where(inside, start[:, None] + col - first[:, None], 0)
    table = torch.where(inside, order[index], 0).to(torch.int32)
    table[:, :shared] = order[:shared]
    return table.cuda(), order[:shared].cuda(), total


def settings(c, gen):
    """Each row's temperature, top-k, top-p and min-p, or None: as the case names
    them, or for "mixed" as a batch of requests has them, some of them greedy."""
    rows, f = c["rows"], c["filters"]
    s = dict.fromkeys(("temperature", "top_k", "top_p", "min_p"))
    t = 0.6 + 0.6 * torch.rand(rows, generator=gen)
    u = torch.rand((4, rows), generator=gen)
    if f == "mixed":
        t[u[0] < 0.1] = 0.0
        s["top_k"] = torch.where(u[1] < 0.5, 0, torch.randint(1, 200, (rows,), generator=gen)).to(torch.int32)
        s["top_p"] = torch.where(u[2] < 0.3, 1.0, 0.8 + 0.19 * torch.rand(rows, generator=gen))
        s["min_p"] = torch.where(u[3] < 0.6, 0.0, 0.1 * torch.rand(rows, generator=gen))
    elif f == "top-k 50, top-p 0.95":
        s["top_k"] = torch.full((rows,), 50, dtype=torch.int32)
        s["top_p"] = torch.full((rows,), 0.95)
    elif f == "top-p 0.9":
        s["top_p"] = torch.full((rows,), 0.9)
    elif f == "min-p 0.05":
        s["min_p"] = torch.full((rows,), 0.05)
    s["temperature"] = t
    return {k: v.cuda() if v is not None else None for k, v in s.items()}


def prepare(case, seed):
    c = dict(case)
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(scale)

    if c["op"] == "sample":
        # logits of a head: a broad body, and a few tokens that the context asks for
        x = normal(c["rows"], c["vocab"], scale=2.2)
        at = torch.randint(0, c["vocab"], (c["rows"], 24), generator=gen, device="cuda")
        x.scatter_(1, at, 4 + 9 * torch.rand(at.shape, generator=gen, device="cuda"))
        s["x"] = x.to(TYPES[c["dtype"]])
        shape = (c["rows"],) if c["draws"] == 1 else (c["rows"], c["draws"])
        s["u"] = torch.rand(shape, generator=gen, device="cuda")
        s.update(settings(c, host))
        s["out"] = torch.empty((c["rows"], c["vocab"]), dtype=torch.float32, device="cuda") if c["probs"] else None
        return s

    dt = TYPES[c["dtype"]]
    held = E4M3 if c["cache"] == "e4m3" else dt
    B, n, hq, hkv, d = c["B"], c["n"], c["hq"], c["hkv"], c["d"]
    s["k_scale"], s["v_scale"] = (0.015, 0.02) if held == E4M3 else (1.0, 1.0)
    s["depth"] = s["words"] = s["counts"] = None
    if c["tree"]:
        s["depth"], s["words"], s["counts"] = (t.cuda() for t in some_trees(B, n, host))
    if c["op"] == "norms":
        # what a projection wrote: q, k and v beside each other, some heads louder
        loud = torch.exp(normal(hq + 2 * hkv, 1, scale=0.7)).to(dt)
        qkv = normal(B, n, hq + 2 * hkv, d, dtype=dt).mul_(loud)
        s["q"], s["k"], s["v"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
        s["wq"], s["wk"] = (1 + normal(d, scale=0.2)).to(TYPES[c["weights"]]), (1 + normal(d, scale=0.2)).to(TYPES[c["weights"]])
        past = torch.full((B,), c["past"], dtype=torch.int64)
        if c["past"]:
            past -= torch.randint(0, 1 + c["past"] // 2, (B,), generator=host)
        # only the pages that this step writes: nothing else is touched
        s["table"], _, pages = paged(c["page"], past, past + n, 0, host)
        s["lens"] = past.to(torch.int32).cuda()
        inv, s["factor"] = frequencies(c["rot"], c["scaling"])
        s["inv_freq"] = inv.cuda()
        s["ck"] = torch.zeros((pages, c["page"], hkv, d), dtype=held, device="cuda")
        s["cv"] = torch.zeros((pages, c["page"], hkv, d), dtype=held, device="cuda")
    else:
        # one sequence has all the tokens of its own, the others fall to none
        each = torch.tensor([c["own"] - (c["own"] * b) // max(1, B - 1) for b in range(B)])[torch.randperm(B, generator=host)]
        lens = c["prefix"] + each
        whole = c["prefix"] // c["page"]
        s["table"], s["pages"], pages = paged(c["page"], torch.full((B,), whole * c["page"]), lens + n, whole, host)
        s["lens"] = lens.to(torch.int32).cuda()
        s["prefix"] = torch.tensor([c["prefix"]], dtype=torch.int32, device="cuda")
        s["q"] = normal(B, n, hq, d, dtype=dt)
        for key, scale in (("ck", s["k_scale"]), ("cv", s["v_scale"])):
            at = torch.empty((pages, c["page"], hkv, d), dtype=held, device="cuda")
            for p0 in range(0, pages, 4096):
                part = normal(min(4096, pages - p0), c["page"], hkv, d, scale=1 / scale)
                at[p0:p0 + 4096] = part.to(held)
            s[key] = at
    if own:
        import verify_gemm_gb300 as vg

        s["cache"] = vg.KVCache(s["ck"], s["cv"], s["table"], s["k_scale"], s["v_scale"])
        if c["op"] == "prefix":
            s["workspace"] = vg.prefix_attention_workspace(s["q"], s["cache"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    if c["op"] == "norms":
        return run_norms(c, s)
    if c["op"] == "prefix":
        return run_prefix(c, s)
    return run_sample(c, s)


def of_cache(t):
    """8-bit codes as the values they stand for (before the scale): exact in bf16."""
    return t.to(torch.bfloat16) if t.dtype == E4M3 else t


EPS = 1e-6


def run_norms(c, s):
    if own:
        import verify_gemm_gb300 as vg

        q = vg.qk_norm_rope_append(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["inv_freq"], s["cache"], s["lens"],
                                   depth=s["depth"], counts=s["counts"], eps=EPS, layout=c["layout"],
                                   factor=s["factor"])
        return q, of_cache(s["ck"]), of_cache(s["cv"])
    n, rot = c["n"], c["rot"]
    steps = torch.arange(n, device="cuda")
    at = s["lens"].double()[:, None] + (s["depth"] if c["tree"] else steps[None, :]).double()
    angle = at[:, :, None] * s["inv_freq"]
    cos, sin = ((f(angle) * s["factor"]).float()[:, :, None, :] for f in (torch.cos, torch.sin))

    def turned(x, w):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        if c["layout"] == "half":
            x1, x2 = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat((x1 * cos - x2 * sin, x1 * sin + x2 * cos), -1)
        else:
            x1, x2 = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack((x1 * cos - x2 * sin, x1 * sin + x2 * cos), -1).flatten(-2)
        return torch.cat((y, x[..., rot:]), -1)

    def held(x, scale, dtype):
        return (x / scale).clamp(-448, 448).to(dtype) if dtype == E4M3 else x.to(dtype)

    slot = s["lens"].long()[:, None] + steps
    page = torch.gather(s["table"].long(), 1, slot // c["page"])
    used = steps[None, :] < (s["counts"][:, None] if s["counts"] is not None else torch.full_like(s["lens"], n)[:, None])
    q, k, v = turned(s["q"], s["wq"]), turned(s["k"], s["wk"]), s["v"].float()
    if s["counts"] is not None:
        page, slot, k, v = page[used], slot[used], k[used], v[used]
        q = torch.where(used[:, :, None, None], q, 0.0)
    # written as bytes: 8-bit floats have no indexed store of their own
    whole = torch.int8 if s["ck"].dtype == E4M3 else torch.int16
    s["ck"].view(whole)[page, slot % c["page"]] = held(k, s["k_scale"], s["ck"].dtype).view(whole)
    s["cv"].view(whole)[page, slot % c["page"]] = held(v, s["v_scale"], s["cv"].dtype).view(whole)
    return q.to(s["q"].dtype), of_cache(s["ck"]), of_cache(s["cv"])


def run_prefix(c, s):
    B, n, hq, hkv, d, page = c["B"], c["n"], c["hq"], c["hkv"], c["d"], c["page"]
    if own:
        import verify_gemm_gb300 as vg

        lse = torch.empty((B, n, hq), dtype=torch.float32, device="cuda")
        out = vg.prefix_attention(s["q"], s["cache"], s["lens"], s["prefix"], s["pages"], tree=s["words"],
                                  counts=s["counts"], lse=lse, workspace=s["workspace"])
        return out, lse
    whole = s["pages"].shape[0]
    rest = (s["table"].shape[1] - whole) * page                   # slots behind the shared pages
    steps = torch.arange(n, device="cuda")
    counts = s["counts"] if s["counts"] is not None else torch.full_like(s["lens"], n)

    def dense(cache, table, scale):  # [..., hkv, slots, d]
        t = cache[table.long()].float().mul_(scale)
        return t.reshape(*table.shape[:-1], table.shape[-1] * page, hkv, d).transpose(-3, -2)

    q = s["q"].float().mul_(d ** -0.5).reshape(B, n, hkv, hq // hkv, d).permute(2, 0, 1, 3, 4)  # [hkv, B, n, group, d]
    rows = n * (hq // hkv)
    shared = torch.matmul(q.reshape(hkv, B * rows, d), dense(s["ck"], s["pages"], s["k_scale"]).transpose(1, 2))
    key = torch.arange(rest, device="cuda")
    draft = whole * page + key[None, :] - s["lens"][:, None]                    # [B, slots]
    if s["words"] is None:
        seen = draft[:, None, :] <= steps[None, :, None]
    else:
        seen = (s["words"][:, :, None] >> draft.clamp(0, 63)[:, None, :]) & 1 == 1
    used = (steps[None, :] < counts[:, None])[:, :, None]
    seen = torch.where(draft[:, None, :] < 0, True, seen) & (draft < counts[:, None])[:, None, :] & used
    seen = seen[:, None, :, None, :].expand(B, 1, n, hq // hkv, rest).reshape(B, 1, rows, rest)
    mine = torch.matmul(q.transpose(0, 1).reshape(B, hkv, rows, d),
                        dense(s["ck"], s["table"][:, whole:], s["k_scale"]).transpose(2, 3))
    mine = mine.masked_fill_(~seen, -math.inf).transpose(0, 1).reshape(hkv, B * rows, rest)
    top = mine.amax(-1, keepdim=True)
    if whole:
        top = torch.maximum(top, shared.amax(-1, keepdim=True))
    top = torch.where(top == -math.inf, 0.0, top)
    shared.sub_(top).exp_()
    mine.sub_(top).exp_()
    total = shared.sum(-1, keepdim=True) + mine.sum(-1, keepdim=True)
    held = (draft < counts[:, None])[:, None, :, None]
    value = torch.where(held, dense(s["cv"], s["table"][:, whole:], s["v_scale"]), 0.0)         # [B, hkv, slots, d]
    o = torch.matmul(mine.reshape(hkv, B, rows, rest), value.transpose(0, 1)).reshape(hkv, B * rows, d)
    o = (o + torch.matmul(shared, dense(s["cv"], s["pages"], s["v_scale"]))) / total
    lse = torch.log(total) + top

    def back(x):
        return x.reshape(hkv, B, n, hq // hkv, -1).permute(1, 2, 0, 3, 4).reshape(B, n, hq, -1)

    # nodes that a tree does not use see nothing
    out = torch.where(used[..., None], back(o), 0.0).to(s["q"].dtype)
    return out, torch.where(used, back(lse)[..., 0], -math.inf)


def run_sample(c, s):
    if own:
        import verify_gemm_gb300 as vg

        tokens = vg.sample(s["x"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                           min_p=s["min_p"], out=s["out"])
        return (tokens, s["out"]) if c["probs"] else tokens
    # in 64 bits: which tokens are kept, and which is drawn, is a comparison of sums
    x = s["x"].double()
    t = s["temperature"].double()[:, None]
    greedy = t <= 0
    w = torch.exp((x - x.amax(-1, keepdim=True)) / torch.where(greedy, 1.0, t))
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices       # ties: the lowest index first
    ws = torch.gather(w, 1, order)
    rank = torch.arange(c["vocab"], device="cuda")[None, :]
    keep = torch.where(greedy, rank < 1, True)
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        keep = keep & ((k <= 0) | (rank < k))
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        among = torch.where(keep, ws, 0.0)
        sums = among.cumsum(-1)
        keep = keep & ((p >= 1) | (sums - among < p * sums[:, -1:]))
    if s["min_p"] is not None:
        keep = keep & (ws >= s["min_p"].double()[:, None])
    kept = torch.zeros_like(keep).scatter_(1, order, keep | (rank == 0))
    w = torch.where(kept, w, 0.0)
    sums = w.cumsum(-1)
    u = s["u"].double().reshape(c["rows"], -1)
    tokens = torch.searchsorted(sums, u * sums[:, -1:], right=True).clamp_(max=c["vocab"] - 1)
    tokens = tokens.to(torch.int32).reshape(s["u"].shape)
    return (tokens, (w / w.sum(-1, keepdim=True)).float()) if c["probs"] else tokens


# ---------------------------------------------------------------- what it takes

def work(case):
    c = case
    if c["op"] == "sample":
        size = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": c["rows"] * (c["vocab"] * (size + (4 if c["probs"] else 0)) + 8 * c["draws"]),
                "flops": 4 * c["rows"] * c["vocab"]}
    held = 1 if c["cache"] == "e4m3" else 2
    if c["op"] == "norms":
        tokens = c["B"] * c["n"]
        return {"bytes": tokens * c["d"] * (4 * c["hq"] + (2 + held) * 2 * c["hkv"]),
                "flops": tokens * (3 * c["rot"] + 4 * c["d"]) * (c["hq"] + c["hkv"])}
    B, n = c["B"], c["n"]
    whole = c["prefix"] // c["page"] * c["page"]
    mine = sum(c["prefix"] - whole + c["own"] - (c["own"] * b) // max(1, B - 1) + n for b in range(B))
    return {"bytes": 2 * (whole + mine) * c["hkv"] * c["d"] * held + B * n * c["hq"] * (4 * c["d"] + 4),
            "flops": 4 * (B * whole + mine) * c["hq"] * n * c["d"]}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    if c["op"] == "norms":
        return exact_norms(c, s)
    if c["op"] == "prefix":
        return exact_prefix(c, s)
    return exact_sample(c, s)


def exact_norms(c, s):
    """The rotation as a product of complex numbers, the append sequence by sequence."""
    B, n, rot = c["B"], c["n"], c["rot"]
    depth = s["depth"] if c["tree"] else torch.arange(n, device="cuda").expand(B, n)
    position = (s["lens"].long()[:, None] + depth.long()).double()
    turn = torch.polar(torch.full((B, n, 1, rot // 2), s["factor"], dtype=torch.float64, device="cuda"),
                       (position[:, :, None] * s["inv_freq"])[:, :, None, :])
    pairs = (slice(0, rot // 2), slice(rot // 2, rot)) if c["layout"] == "half" else (slice(0, rot, 2), slice(1, rot, 2))

    def turned(x, w):
        x = x.double()
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["d"] + EPS) * w.double()
        z = torch.complex(x[..., pairs[0]], x[..., pairs[1]]) * turn
        x[..., pairs[0]], x[..., pairs[1]] = z.real, z.imag
        return x

    q, k, v = turned(s["q"], s["wq"]), turned(s["k"], s["wk"]) / s["k_scale"], s["v"].double() / s["v_scale"]
    counts = s["counts"].tolist() if s["counts"] is not None else [n] * B
    lens, table, page = s["lens"].tolist(), s["table"].long(), c["page"]
    for b in range(B):
        q[b, counts[b]:] = 0
    if c["cache"] == "e4m3":  # a code is a choice between neighbours: a value that it stands for has no 64-bit form
        return q, None, None
    ck, cv = (torch.zeros(s[key].shape, dtype=torch.float64, device="cuda") for key in ("ck", "cv"))
    for b in range(B):
        slot = torch.arange(lens[b], lens[b] + counts[b], device="cuda")
        at = table[b, slot // page], slot % page
        ck[at], cv[at] = k[b, :counts[b]], v[b, :counts[b]]
    return q, ck, cv


def exact_prefix(c, s):
    """Sequence by sequence over its own page table, as if nothing were shared, some rows at a time."""
    B, n, hq, hkv, d = c["B"], c["n"], c["hq"], c["hkv"], c["d"]
    if 4 * B * n * hq * (c["prefix"] + c["own"]) * d > 5e12:
        return None
    out = torch.zeros((B, n, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, n, hq), -math.inf, dtype=torch.float64, device="cuda")
    lens = s["lens"].tolist()
    counts = s["counts"].tolist() if s["counts"] is not None else [n] * B
    for b in range(B):
        slot = torch.arange(lens[b] + counts[b], device="cuda")
        at = s["table"][b].long()[slot // c["page"]], slot % c["page"]
        see = torch.ones((counts[b], lens[b] + counts[b]), dtype=torch.bool, device="cuda")
        if c["tree"]:
            bits = [[(int(w) >> j) & 1 for j in range(counts[b])] for w in s["words"][b, :counts[b]].tolist()]
            see[:, lens[b]:] = torch.tensor(bits, device="cuda").bool()
        else:
            see[:, lens[b]:] = torch.ones((counts[b], counts[b]), device="cuda").tril().bool()
        for g in range(hkv):
            k = s["ck"][at[0], at[1], g].double() * s["k_scale"]
            v = s["cv"][at[0], at[1], g].double() * s["v_scale"]
            heads = slice(g * (hq // hkv), (g + 1) * (hq // hkv))
            x = torch.einsum("ihd,jd->hij", s["q"][b, :counts[b], heads].double(), k) / math.sqrt(d)
            x = torch.where(see[None], x, -math.inf)
            norm = torch.logsumexp(x, -1)
            out[b, :counts[b], heads] = torch.einsum("hij,jd->ihd", torch.exp(x - norm[..., None]), v)
            lse[b, :counts[b], heads] = norm.T
    return out, lse


def exact_sample(c, s):
    """Row by row over the groups of equal logits: how many tokens are kept, then
    which, then the draw."""
    u = s["u"].double().reshape(c["rows"], -1)
    tokens, rows = torch.zeros(u.shape, dtype=torch.int32), []
    for r in range(c["rows"]):
        x = s["x"][r].double()
        t = float(s["temperature"][r])
        value, size = torch.unique(-x, return_counts=True)          # largest logit first
        value = -value
        weight = torch.exp((value - value[0]) / t) if t > 0 else (value == value[0]).double()
        before = torch.cumsum(size, 0) - size
        k = int(s["top_k"][r]) if s["top_k"] is not None else 0
        k = 1 if t <= 0 else k if k > 0 else c["vocab"]
        taken = (k - before).clamp(min=0).minimum(size)             # of each group
        keep = k
        p = float(s["top_p"][r]) if s["top_p"] is not None else 1.0
        if p < 1:
            mass = torch.cumsum(weight * taken, 0)
            target = p * float(mass[-1])
            g = int((mass < target).sum())
            left = target - (float(mass[g - 1]) if g else 0.0)
            keep = min(keep, int(before[g]) + max(1, min(int(taken[g]), math.ceil(left / float(weight[g])))))
        if s["min_p"] is not None:
            keep = min(keep, max(1, int(size[weight >= float(s["min_p"][r])].sum())))
        g = int((before < keep).sum()) - 1                          # the last group with a token that is kept
        mask = x > value[g]
        mask[(x == value[g]).nonzero()[:keep - int(before[g]), 0]] = True
        e = torch.where(mask, torch.exp((x - value[0]) / (t if t > 0 else 1.0)), 0.0)
        sums = torch.cumsum(e, 0)
        tokens[r] = ((sums[None, :] <= u[r][:, None] * sums[-1]).sum(-1)).clamp(max=c["vocab"] - 1).cpu()
        if c["probs"]:
            rows.append(e / e.sum())
    tokens = tokens.reshape(s["u"].shape)
    return (tokens, torch.stack(rows)) if c["probs"] else tokens
