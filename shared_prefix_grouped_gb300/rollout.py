"""Generating the responses of shared-prefix groups with the decoder layer of layer.py, composed from
the library's C-ABI kernels.  Torch allocates, and counts the generated tokens.

    r = Rollout(prefix_lens, group_sizes, heads_q, heads_kv, head_dim, max_new, device="cuda")
    caches = [r.cache() for _ in layers]                      # (k_cache, v_cache) of each layer
    x = layer_prefill(r, r.prefix_layout(), x_prefix, *weights, *caches[i], ...)  # once per layer
    for each token:
        x = layer_decode(r, x, *weights, *caches[i], ...)     # [responses, hidden], per layer
        logits = api.gemm_bf16(norm(x), w_head)
        tokens, logprobs = api.sample(logits, u, temperature=t, top_p=p)
        r.advance()

Every group's prefix is kept once, in pages that its responses share; a response's own keys and values
go to pages of its own.  One plan serves every layer and every step (the number of keys a response
has is read on the device), so a step of all layers can be captured into a CUDA graph, advance()
included.  With cache_dtype=torch.float8_e4m3fn the caches take half the memory: 8-bit codes with a
scale per 16 slots and head, which the same two functions append to and attend to.
"""
from __future__ import annotations

from typing import Optional, Sequence

import torch

from . import api
from .layer import _gains, layer_fwd


class Rollout:
    """Page tables, plan, workspace and counters of one batch of groups under generation.

    A response holds up to max_new tokens, rounded up to whole pages.  A step beyond stores nothing and
    attends to the keys there are; it is recorded and told by api.device_status().  A response that has
    ended may be parked: with cache_pos[s] = own_lens[s] = -2**30 its tokens are stored nowhere and its
    own keys are not read any more, and advance() leaves it so; its rows of the layer's output are
    then of no use.  layer_prefill and layer_decode compute in bf16; with dtype float32 the caches, page
    tables and plan serve api.cache_append and api.decode_attn.  cache_dtype (default: dtype) may be
    torch.float8_e4m3fn: then cache() gives a pair of api.ScaledCache, for the functions' _e4m3 forms."""

    def __init__(self, prefix_lens: Sequence[int], group_sizes: Sequence[int], heads_q: int,
                 heads_kv: int, head_dim: int, max_new: int, *, page_size: int = 64,
                 dtype: torch.dtype = torch.bfloat16, cache_dtype: Optional[torch.dtype] = None,
                 device="cuda"):
        device = torch.device(device)
        cache_dtype = dtype if cache_dtype is None else cache_dtype
        if cache_dtype not in (dtype, torch.float8_e4m3fn):
            raise ValueError(f"cache_dtype must be {dtype} or torch.float8_e4m3fn, got {cache_dtype}")
        if cache_dtype is torch.float8_e4m3fn and page_size % api.CACHE_BLOCK:
            raise ValueError(f"a cache in 8 bits takes a page_size of whole blocks of {api.CACHE_BLOCK}")
        if max_new < 1:
            raise ValueError("max_new must be at least 1")
        self.prefix_lens, self.group_sizes = list(prefix_lens), list(group_sizes)
        self.heads_q, self.heads_kv, self.head_dim = heads_q, heads_kv, head_dim
        self.max_new, self.page_size, self.dtype = max_new, page_size, dtype
        self.cache_dtype = cache_dtype
        own = (max_new + page_size - 1) // page_size
        self.plan = api.plan_decode(prefix_lens, group_sizes, heads_q, heads_kv, head_dim, page_size,
                                    own, dtype, device)
        self.device = device = self.plan.tables.device
        self.workspace = api.decode_workspace(self.plan, cache_dtype)
        S, B = self.plan.num_seqs, len(self.prefix_lens)
        width = max(max((n + page_size - 1) // page_size for n in self.prefix_lens), 1)
        self.num_pages = B * width + S * own
        table = torch.arange(self.num_pages, dtype=torch.int32, device=device)
        self.prefix_pages = table[:B * width].view(B, width)
        self.own_pages = table[B * width:].view(S, own)
        # The next token of response s is its own key cache_pos[s], at position positions[s]; with it
        # the response has own_lens[s] keys of its own.
        self.cache_pos = torch.zeros(S, dtype=torch.int32, device=device)
        self.own_lens = torch.ones(S, dtype=torch.int32, device=device)
        first = [n for n, g in zip(self.prefix_lens, self.group_sizes) for _ in range(g)]
        self.positions = torch.tensor(first, dtype=torch.int32, device=device)

    def cache(self):
        """(k_cache, v_cache) of one layer."""
        if self.cache_dtype is torch.float8_e4m3fn:
            return tuple(api.scaled_cache(self.num_pages, self.page_size, self.heads_kv, self.head_dim,
                                          self.device) for _ in range(2))
        shape = (self.num_pages, self.page_size, self.heads_kv, self.head_dim)
        return tuple(torch.empty(shape, dtype=self.dtype, device=self.device) for _ in range(2))

    def append(self, *args, **kw):
        """api.cache_append for this rollout's caches."""
        eight = self.cache_dtype is torch.float8_e4m3fn
        return (api.cache_append_e4m3 if eight else api.cache_append)(*args, **kw)

    def attn(self, q, k_cache, v_cache):
        """api.decode_attn of a step's queries for this rollout's caches."""
        eight = self.cache_dtype is torch.float8_e4m3fn
        return (api.decode_attn_e4m3 if eight else api.decode_attn)(
            self.plan, q, k_cache, v_cache, self.prefix_pages, self.own_pages, self.own_lens,
            workspace=self.workspace)

    def advance(self) -> None:
        """The step's token is done: every response's next one follows it."""
        self.cache_pos += 1
        self.own_lens += 1
        self.positions += 1

    def prefix_layout(self) -> api.Layout:
        """The prefixes as a packed batch without responses, for layer_prefill."""
        B = len(self.prefix_lens)
        lay = api.pack(self.prefix_lens, [0] * B, [], self.device)
        lay.page_rows = torch.repeat_interleave(
            torch.arange(B, dtype=torch.int32), torch.tensor(self.prefix_lens)).to(self.device)
        return lay


def layer_prefill(rollout: Rollout, layout: api.Layout, x, w_qkv, w_o, w_gu, w_d, g1, g2, k_cache,
                  v_cache, *, rope_theta, eps, g_q: Optional[torch.Tensor] = None,
                  g_k: Optional[torch.Tensor] = None):
    """The layer over the packed prefixes x [sum of prefix_lens, hidden] (layout =
    rollout.prefix_layout()), whose rotated keys and whose values go to the prefixes' pages."""
    _gains(g_q, g_k)
    Hq, Hkv, d = rollout.heads_q, rollout.heads_kv, rollout.head_dim
    y, saved = layer_fwd(layout, x, w_qkv, w_o, w_gu, w_d, g1, g2, heads_q=Hq, heads_kv=Hkv,
                         head_dim=d, rope_theta=rope_theta, eps=eps, g_q=g_q, g_k=g_k)
    T = x.shape[0]
    rollout.append(saved["k"].view(T, Hkv, d), saved["v"].view(T, Hkv, d), k_cache, v_cache,
                   rollout.prefix_pages, layout.position_ids, page_rows=layout.page_rows)
    return y


def layer_decode(rollout: Rollout, x, w_qkv, w_o, w_gu, w_d, g1, g2, k_cache, v_cache, *, rope_theta,
                 eps, g_q: Optional[torch.Tensor] = None, g_k: Optional[torch.Tensor] = None):
    """The layer for the next token of every response, x [responses, hidden]: appends its key and
    value, attends to the shared prefix and the response's own keys, and returns y like x."""
    norms = _gains(g_q, g_k)
    r, bf = rollout, torch.bfloat16
    Hq, Hkv, d = r.heads_q, r.heads_kv, r.head_dim
    S = x.shape[0]
    h1, _, _ = api.rmsnorm_fwd(x, g1, eps)
    qkv = api.gemm_bf16(h1, w_qkv, out_dtype=bf).view(S, Hq + 2 * Hkv, d)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if norms:
        q, k = api.qk_norm_rope_fwd(q, k, g_q, g_k, eps, r.positions, rope_theta=rope_theta)
        r.append(k, v, k_cache, v_cache, r.own_pages, r.cache_pos)
    else:
        q = r.append(k, v, k_cache, v_cache, r.own_pages, r.cache_pos, q=q, positions=r.positions,
                     rope_theta=rope_theta)
    o, _ = r.attn(q, k_cache, v_cache)
    a = api.gemm_bf16(o.view(S, Hq * d), w_o, out_dtype=bf)
    h2, x2, _ = api.rmsnorm_fwd(x, g2, eps, residual=a)
    act = api.swiglu_fwd(api.gemm_bf16(h2, w_gu, out_dtype=bf))
    y = x2.clone()
    api.gemm_bf16(act, w_d, out=y, accumulate=True)
    return y
