"""The operators of a verify round between and behind its products: rotary
positions with the append to a paged cache (and norms of the heads before it),
attention of a tree of drafted tokens over that cache (and behind a prefix that a
batch shares), the probabilities of logits, draws from truncated distributions
of them and the verification of the drafted tokens.

Every step runs in the CUDA kernels of ``libvgemm.so``.  The calls go through
``_vgtorch.so``, which checks the tensors, allocates the outputs and calls the
C ABI.  Lengths, node counts and page tables are read on the device, so a
captured graph serves every length.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from ._lib import (VG_ROPE_HALF, VG_ROPE_INTERLEAVED, VG_TYPE_BF16, VG_TYPE_E4M3, VG_TYPE_FP16,
                   vg_kv_cache)

_TYPES = {torch.bfloat16: VG_TYPE_BF16, torch.float16: VG_TYPE_FP16,
          torch.float8_e4m3fn: VG_TYPE_E4M3}
_LAYOUTS = {"half": VG_ROPE_HALF, "interleaved": VG_ROPE_INTERLEAVED}
_native = None


def _calls():
    global _native
    if _native is None:
        _native = _lib.load_torch()
    return _native


def _on(stream, tensor):
    """Makes the stream current; it has to be of the tensors' device."""
    if stream.device != getattr(tensor, "device", None):
        raise ValueError("the stream and the tensors are on different devices")
    return torch.cuda.stream(stream)


def _checked(result, where):
    if type(result) is int:          # a vg_status
        _lib.check(result, where)
    return result


class KVCache:
    """A paged key/value cache: k and v [pages, page_size, heads, head_dim]
    (views of other orders are fine, the last dimension contiguous) in
    bfloat16, float16 or float8_e4m3fn, and page_table int32 [batch,
    max_pages]; slot s of sequence b is token s % page_size of page
    page_table[b, s // page_size].  An 8-bit code is worth k_scale (v_scale)
    times its value.  The tensors are kept alive and read at every call; the
    table's contents may change between calls."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor,
                 k_scale: float = 1.0, v_scale: float = 1.0):
        for t, name in ((k, "k"), (v, "v")):
            if not t.is_cuda or t.dim() != 4 or t.dtype not in _TYPES or t.stride(3) != 1:
                raise ValueError(f"{name}: expected a CUDA tensor [pages, page_size, heads, "
                                 "head_dim] whose last dimension is contiguous")
        if k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v must have the same shape, type and device")
        if not (page_table.device == k.device and page_table.dtype == torch.int32
                and page_table.dim() == 2 and (page_table.stride(1) == 1 or page_table.shape[1] == 1)):
            raise ValueError("page_table: expected a CUDA int32 tensor [batch, max_pages]")
        self.k, self.v, self.page_table = k, v, page_table
        self.batch, self.heads, self.head_dim, self.dtype = (page_table.shape[0], k.shape[2],
                                                             k.shape[3], k.dtype)
        c = vg_kv_cache()
        c.k, c.v, c.page_table = k.data_ptr(), v.data_ptr(), page_table.data_ptr()
        c.type, c.heads, c.head_dim, c.page_size = _TYPES[k.dtype], k.shape[2], k.shape[3], k.shape[1]
        c.pages = k.shape[0]
        for i, dim in enumerate((0, 1, 2)):
            # the stride of a dimension of one is arbitrary: any legal one will do
            c.k_stride[i] = k.stride(dim) if k.shape[dim] > 1 else 256
            c.v_stride[i] = v.stride(dim) if v.shape[dim] > 1 else 256
        c.batch, c.max_pages = page_table.shape
        c.table_stride = page_table.stride(0) if c.batch > 1 else c.max_pages
        c.k_scale, c.v_scale = k_scale, v_scale
        _lib.check(_lib.vg_kv_cache_init(ctypes.byref(c)), "vg_kv_cache_init")
        self._c = c
        self._at = ctypes.addressof(c)
        self._device = k.device.index


def rope_frequencies(rot: int, base: float = 10000.0, scaling: str | None = None,
                     factor: float = 1.0, context: int = 0, beta_fast: float = 32.0,
                     beta_slow: float = 1.0, device="cuda"):
    """(inv_freq float64 [rot / 2], attention factor) for rope_append.

    inv_freq[j] = base ** (-2 j / rot).  scaling "linear" divides all of them
    by `factor`; "ntk" raises the base so that the slowest pair is divided by
    it; "yarn" leaves the pairs that turn more than beta_fast times in the
    original `context`, divides those that turn less than beta_slow times, and
    goes over evenly in the logarithm of the turns between the two, with the
    attention factor 0.1 ln(factor) + 1.  The ramp's ends are taken as they come
    out; a model trained with a table whose ramp begins and ends at whole pairs
    (some percent apart within the ramp) needs that table as inv_freq."""
    if rot < 2 or rot % 2 or base <= 1 or factor < 1:
        raise ValueError("rot must be even and positive, base > 1 and factor >= 1")
    j = torch.arange(rot // 2, dtype=torch.float64)
    m = 1.0
    if scaling == "ntk":
        if rot < 4:
            raise ValueError("ntk scaling needs rot >= 4")
        base = base * factor ** (rot / (rot - 2))
    inv = base ** (-2.0 * j / rot)
    if scaling == "linear":
        inv = inv / factor
    elif scaling == "yarn":
        if context < 1 or not beta_fast > beta_slow > 0:
            raise ValueError("yarn scaling needs the original context and beta_fast > beta_slow > 0")
        turns = context * inv / (2 * math.pi)
        keep = ((torch.log(turns) - math.log(beta_slow))
                / (math.log(beta_fast) - math.log(beta_slow))).clamp(0, 1)
        inv = inv * keep + inv / factor * (1 - keep)
        m = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError("scaling: None, 'linear', 'ntk' or 'yarn'")
    return inv.to(device), m


def rope_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, inv_freq: torch.Tensor,
                cache: KVCache, lens: torch.Tensor, depth: torch.Tensor | None = None,
                counts: torch.Tensor | None = None, layout: str = "half", factor: float = 1.0,
                q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rotates q [batch, n, q_heads, head_dim] and k, and appends k and v
    [batch, n, heads, head_dim] to the cache; returns the rotated q.

    Node i of sequence b goes to slot lens[b] + i and has position lens[b] +
    depth[b, i] (depth None: i).  The first 2 * inv_freq.numel() elements of a
    head turn: pairs (j, j + rot/2) for layout "half", (2j, 2j + 1) for
    "interleaved".  Nodes past counts[b] append nothing and give 0."""
    if stream is not None:
        with _on(stream, q):                 # q_out, too, is made there
            return rope_append(q, k, v, inv_freq, cache, lens, depth, counts, layout, factor, q_out)
    if layout not in _LAYOUTS:
        raise ValueError("layout: 'half' or 'interleaved'")
    return _checked((_native or _calls()).rope_append(
        q, k, v, inv_freq, cache._at, lens, depth, counts, _LAYOUTS[layout], factor, q_out,
        cache._device),
        "vg_rope_append")


def qk_norm_rope_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                        q_weight: torch.Tensor | None, k_weight: torch.Tensor | None,
                        inv_freq: torch.Tensor, cache: KVCache, lens: torch.Tensor,
                        depth: torch.Tensor | None = None, counts: torch.Tensor | None = None,
                        eps: float = 1e-6, layout: str = "half", factor: float = 1.0,
                        q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """rope_append of q and k whose heads are normed first, in the same launch:
    x * weight / sqrt(mean(x ** 2) + eps) over each whole head, in float32 up to
    what is stored.  q_weight, k_weight [head_dim]: float32 or q's type, both the
    same, None: ones.  eps at least 2 ** -126."""
    if stream is not None:
        with _on(stream, q):
            return qk_norm_rope_append(q, k, v, q_weight, k_weight, inv_freq, cache, lens, depth, counts, eps,
                                       layout, factor, q_out)
    if layout not in _LAYOUTS:
        raise ValueError("layout: 'half' or 'interleaved'")
    return _checked((_native or _calls()).qk_norm_rope_append(
        q, k, v, inv_freq, cache._at, lens, depth, counts, _LAYOUTS[layout], factor, q_out,
        cache._device, q_weight, k_weight, eps), "vg_qk_norm_rope_append")


def tree_attention_workspace(q: torch.Tensor, cache: KVCache) -> torch.Tensor:
    """A zero-filled workspace for tree_attention with q of this shape."""
    if q.device != cache.k.device:
        raise ValueError("q and the cache are on different devices")
    if cache._device != torch.cuda.current_device():
        with torch.cuda.device(cache._device):
            return tree_attention_workspace(q, cache)
    return _workspace("vg_tree_attention_workspace_size", q, cache)


def _workspace(query, q, cache):
    n = ctypes.c_size_t()
    _lib.check(getattr(_lib, query)(q.shape[1], q.shape[2], cache._at, ctypes.byref(n)), query)
    return torch.zeros(n.value, dtype=torch.uint8, device=q.device)


def tree_attention(q: torch.Tensor, cache: KVCache, lens: torch.Tensor,
                   tree: torch.Tensor | None = None, counts: torch.Tensor | None = None,
                   scale: float | None = None, out: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """Attention of q [batch, n, q_heads, head_dim], n <= 64, over the cache.

    Node i of sequence b attends to the lens[b] committed slots and to the
    nodes whose bits are set in tree[b, i] (int64 words; None: a chain), those
    below counts[b] alone.  A node without any key and a node past counts[b]
    give 0.  scale: 1 / sqrt(head_dim) by default.  lse: float32 [batch, n,
    q_heads], written if given.  workspace: from tree_attention_workspace,
    made anew by each call that is given none; calls that share one must not
    overlap.  A wait on the GPU that runs out, which should not happen, gives
    NaN and sets the workspace's error word: while workspace_error has not read
    and cleared it, calls on that workspace give NaN.  (The word of a workspace
    that a call made for itself cannot be read.)"""
    if stream is not None:
        with _on(stream, q):                 # out and a new workspace, too, are made there
            return tree_attention(q, cache, lens, tree, counts, scale, out, lse, workspace)
    if workspace is None:
        workspace = tree_attention_workspace(q, cache)
    return _checked((_native or _calls()).tree_attention(
        q, cache._at, lens, tree, counts, cache.head_dim ** -0.5 if scale is None else scale, out, lse,
        workspace, cache._device), "vg_tree_attention")


def prefix_attention_workspace(q: torch.Tensor, cache: KVCache) -> torch.Tensor:
    """A zero-filled workspace for prefix_attention with q of this shape."""
    if q.device != cache.k.device:
        raise ValueError("q and the cache are on different devices")
    if cache._device != torch.cuda.current_device():
        with torch.cuda.device(cache._device):
            return prefix_attention_workspace(q, cache)
    return _workspace("vg_prefix_attention_workspace_size", q, cache)


def prefix_attention(q: torch.Tensor, cache: KVCache, lens: torch.Tensor, prefix: torch.Tensor,
                     prefix_pages: torch.Tensor, tree: torch.Tensor | None = None,
                     counts: torch.Tensor | None = None, scale: float | None = None,
                     out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """tree_attention of sequences that begin with the same tokens: the pages
    that the prefix fills are read once for the whole batch.

    prefix int32 [1]: its tokens.  Its first prefix // page_size pages (as many as
    prefix_pages, int32 [pages], has at most) are shared; what it has behind
    them lies in each sequence's own pages.  lens counts the prefix's tokens, too, and
    the row of the page table of a sequence that shares has its own pages from
    there on (the entries before are not read).  A sequence shorter than the shared pages has no
    part in them and takes all its slots from its own row.  The result is that of
    tree_attention over tables that begin with the shared pages, but for the
    order of its sums; everything else is as there.  workspace: from
    prefix_attention_workspace."""
    if stream is not None:
        with _on(stream, q):                 # out and a new workspace, too, are made there
            return prefix_attention(q, cache, lens, prefix, prefix_pages, tree, counts, scale, out, lse, workspace)
    if workspace is None:
        workspace = prefix_attention_workspace(q, cache)
    return _checked((_native or _calls()).prefix_attention(
        q, cache._at, lens, tree, counts, cache.head_dim ** -0.5 if scale is None else scale, out, lse,
        workspace, cache._device, prefix, prefix_pages), "vg_prefix_attention")


def probabilities(logits: torch.Tensor, temperature: torch.Tensor | None = None,
                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """float32 softmax over the last dimension of contiguous logits (bfloat16,
    float16 or float32), each row over its own temperature (float32, one for
    every row; None: 1).  A temperature <= 0 gives 1 at the row's first
    largest logit."""
    if stream is not None:
        with _on(stream, logits):
            return probabilities(logits, temperature, out)
    return _checked((_native or _calls()).probabilities(logits, temperature, out), "vg_probabilities")


def sample(logits: torch.Tensor, u: torch.Tensor, temperature: torch.Tensor | None = None,
           top_k: torch.Tensor | None = None, top_p: torch.Tensor | None = None,
           min_p: torch.Tensor | None = None, out: torch.Tensor | None = None,
           stream=None) -> torch.Tensor:
    """Tokens drawn from the softmax of logits [rows, vocab] (bfloat16, float16 or
    float32; rows may lie apart), truncated: int32, one for each number of u
    (float32 [rows] or [rows, draws], in [0, 1)).

    Each row has its own temperature, top_p, min_p (float32) and top_k (int32), or
    all none (None: 1, and no limit).  In the order of the logits, equal ones by
    index, the first top_k tokens are kept (<= 0: all), of these the fewest
    whose probabilities sum to top_p of theirs (>= 1: all), of these the ones
    min_p times as probable as the first; one at least.  The token is the first
    index whose running sum over what is kept exceeds u of the whole.  A
    temperature <= 0 keeps the first largest logit.  A row without a
    distribution (a NaN, or nothing but -infinity) has the token -1.

    out, float32 like logits and contiguous, receives the truncated distribution itself, which
    verify_tree takes as p and, for drafts drawn from it, as q.
    include/vgemm.h (vg_sample) has the rule."""
    if stream is not None:
        with _on(stream, logits):
            return sample(logits, u, temperature, top_k, top_p, min_p, out)
    return _checked((_native or _calls()).sample(logits, u, temperature, top_k, top_p, min_p, out), "vg_sample")


def verify_tree(p: torch.Tensor, q: torch.Tensor | None, tokens: torch.Tensor,
                parents: torch.Tensor, u: torch.Tensor, counts: torch.Tensor | None = None,
                stream=None):
    """Verifies each sequence's drafted tokens: p float32 [batch, n, vocab],
    the target's distribution after each node; q float32 [batch, rows, vocab],
    the distribution each node's children were drafted from, independently of
    one another (with children made distinct, by top-k or by draws without
    replacement, what comes out is not distributed as p); tokens and
    parents int32 [batch, n]; u float32 [batch, n], random numbers in [0, 1).

    Returns int32 (accepted [batch], path [batch, n], out [batch, n + 1]): how
    many drafts hold, their nodes, and their tokens with the one drawn after
    them; -1 behind.  include/vgemm.h (vg_verify_tree) has the rule."""
    if stream is not None:
        with _on(stream, p):
            return verify_tree(p, q, tokens, parents, u, counts)
    return _checked((_native or _calls()).verify_tree(p, q, tokens, parents, u, counts), "vg_verify_tree")
