"""Rounds of speculative decoding with every step in the library.

A small one-layer model verifies chains of drafted tokens for two requests at
once: 2 requests x 4 nodes (the last committed token and 3 drafts) are the 8
columns of each weight-streaming product.  A round is

  embedding -> RMS norm -> q, k, v   one fused pass (VerifyPlan)
  rope_append                        rotates q and k, appends k and v to the paged cache
  tree_attention                     each node over the cache and the nodes before it
  o projection, output head          NVFP4 products
  probabilities                      a temperature for each request
  verify_tree                        which drafts hold, and the token after them

and the committed lengths grow on the device: nothing waits for the host.
Random weights and drafts stand in for a checkpoint and a drafting model.

Run from the repository root on a GB300: ``python examples/verify_round.py``.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch
import verify_gemm_gb300 as vg

torch.manual_seed(0)
dev = "cuda"
B, n = 2, 4                                     # requests, nodes of a chain
H, heads, kv_heads, d, V = 1024, 8, 2, 128, 4096
page, pages = 16, 32


def weight(M, K):
    return vg.nvfp4_pack(torch.randn(M, K, device=dev) * K ** -0.5)


embed = torch.randn(V, H, device=dev).to(torch.bfloat16)
gamma = torch.ones(H, dtype=torch.bfloat16, device=dev)
wq, wk, wv = weight(heads * d, H), weight(kv_heads * d, H), weight(kv_heads * d, H)
wo, head = weight(H, heads * d), weight(V, H)


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16, device=dev)


x, xn = bf16(B * n, H), bf16(B * n, H)
q, k, v = bf16(B * n, heads * d), bf16(B * n, kv_heads * d), bf16(B * n, kv_heads * d)
plan = vg.VerifyPlan([(vg.RMSNorm(gamma), x, xn, 0), (wq, xn, q, 1, True), (wk, xn, k, 1, True),
                      (wv, xn, v, 1, True)], B * n)

# the cache: pages in any order, each request's own
table = torch.randperm(2 * pages, device=dev).to(torch.int32).view(B, pages)
cache = vg.KVCache(bf16(2 * pages, page, kv_heads, d), bf16(2 * pages, page, kv_heads, d), table)
lens = torch.zeros(B, dtype=torch.int32, device=dev)
inv_freq, factor = vg.rope_frequencies(d, base=1e6, scaling="yarn", factor=4.0, context=32768)
q4 = q.view(B, n, heads, d)
workspace = vg.tree_attention_workspace(q4, cache)
temperature = torch.tensor([0.0, 0.8], device=dev).repeat_interleave(n)    # greedy, and sampled
parents = torch.arange(-1, n - 1, dtype=torch.int32, device=dev).expand(B, n).contiguous()

tokens = torch.randint(0, V, (B, n), dtype=torch.int32, device=dev)        # node 0: the last token
batch = torch.arange(B, device=dev)
for step in range(4):
    drafts = torch.softmax(torch.randn(B, n - 1, V, device=dev), -1)       # the drafting model's rows
    tokens[:, 1:] = torch.multinomial(drafts.view(-1, V), 1).view(B, n - 1).to(torch.int32)
    x.copy_(embed[tokens.view(-1).long()])
    plan.run()
    qr = vg.rope_append(q4, k.view(B, n, kv_heads, d), v.view(B, n, kv_heads, d), inv_freq, cache, lens,
                        factor=factor)
    att = vg.tree_attention(qr, cache, lens, workspace=workspace)
    y = vg.gemv(wo, att.view(B * n, heads * d))
    logits = vg.gemv(head, y)
    p = vg.probabilities(logits, temperature=temperature).view(B, n, V)
    accepted, path, out = vg.verify_tree(p, drafts, tokens, parents, torch.rand(B, n, device=dev))
    # the accepted nodes of a chain lie in the cache behind the committed tokens already
    lens += 1 + accepted
    tokens[:, 0] = out[batch, accepted.long()]
    print(f"round {step}: accepted {accepted.tolist()}, out {out.tolist()}, lengths {lens.tolist()}")
assert plan.check() == 0 and vg.workspace_error(workspace) == 0

# the last round's attention against PyTorch arithmetic on the cache
past = int(lens[1] - 1 - accepted[1])
slot = torch.arange(past + n, device=dev)
at = table[1].long()[slot // page], slot % page
kk = cache.k[at].float().repeat_interleave(heads // kv_heads, 1)
vv = cache.v[at].float().repeat_interleave(heads // kv_heads, 1)
s = torch.einsum("nhd,shd->hns", qr[1].float(), kk) * d ** -0.5
s.masked_fill_(slot[None, :] > past + torch.arange(n, device=dev)[:, None], float("-inf"))
ref = torch.einsum("hns,shd->nhd", torch.softmax(s, -1), vv)
err = (att[1].float() - ref).abs().max().item()
print(f"attention: largest difference {err:.1e} (BF16 output)")
assert err < 2e-2
plan.close()
