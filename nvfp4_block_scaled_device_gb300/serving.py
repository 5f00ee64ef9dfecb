"""A serving step of decoder layers over a paged KV cache, as one launch set.

A step has R requests with q_len[r] new tokens each (whole prompts, chunks of
them, single tokens of decoding, mixed) behind ctx_len[r] cached ones.  Once
per step (``AttnPlan``):

    positions, cache slots, block table, attention schedule   nvfp4_attn_plan

and per layer, for the T packed new tokens (hidden H, heads of D columns):

    h        = NVFP4(RMSNorm(x; attn_norm))
    q, k, v  = h @ Wqkv^T, q and k rotated at the plan's positions
    cache   <- k, v                                             nvfp4_kv_append
    a        = NVFP4(attention of q over the cache)             nvfp4_attn_paged

or, where the model normalises its query and key heads (q_norm, k_norm) or pairs
the halves of a head, norm, rotation and the write of the cache in one pass
behind the projection (nvfp4_qk_norm_rope).  The cache may be one in 4 bits
(KVCache4): nvfp4_kv4_append, nvfp4_attn_paged4.  Then

    x1       = x + a @ Wo^T
    out      = x1 + MLP(x1)

The lengths stay on the device and nothing waits for the host, so a step can
be captured in a CUDA graph and replayed as the contexts grow (plan.cursor counts the pages taken):

    layer = ServingLayer(plan, cache, weights, attn_norm, mlp_norm, cos_t, sin_t)
    with torch.cuda.graph(graph):
        nvfp4_attn_plan(plan, q_len, ctx_len, free_pages, plan.cursor)
        layer.forward(x, out)                 # and the other layers
        ctx_len.add_(q_len)

Requests that fork, end, or whose pages are moved together: nvfp4_pages_fork,
nvfp4_pages_free and nvfp4_pages_copy on the same block table and ctx_len, between
steps (PageTable).  Each gives the cursor or the free list that the next step's
nvfp4_attn_plan takes.

Plans of different sizes (prompts, decoding) that share the block table, and
layers that share the cache, serve the same requests.  Each plan has a cursor of
its own: where the next step is another plan's, its cursor is copied first
(decode.cursor.copy_(prompts.cursor)), or pages are given out twice.

A plan without a cache (page_size 0) runs packed prompts by themselves
(nvfp4_attn_prompt), e.g. for embeddings or scores.
"""
from __future__ import annotations

import torch

from . import (NVFP4_INTER_DYNAMIC, AttnPlan, KVCache, KVCache4, NVFP4Tensor, attn_workspace_bytes,
               gemm_workspace_bytes, mlp_workspace_bytes, nvfp4_attn_paged, nvfp4_attn_paged4, nvfp4_attn_prompt,
               nvfp4_gemm, nvfp4_gemm_rope, nvfp4_kv4_append, nvfp4_kv_append, nvfp4_mlp, nvfp4_qk_norm_rope,
               nvfp4_scale_quantize, workspace)

_PASS_ROWS = 32      # rows of a request that nvfp4_attn_paged4 takes in one pass over its keys' codes


class ServingLayer:
    """One layer's buffers, all allocated at construction (layers that run one
    after the other may share ``scratch`` of an earlier one of the same sizes; the
    attention's workspace alone is 40 MB)."""

    def __init__(self, plan: AttnPlan, cache: KVCache | KVCache4 | None, weights: dict, attn_norm: torch.Tensor,
                 mlp_norm: torch.Tensor, cos_t: torch.Tensor, sin_t: torch.Tensor, eps=1e-6, scratch=None,
                 q_norm: torch.Tensor | None = None, k_norm: torch.Tensor | None = None, halves=False, expand=True):
        """weights: NVFP4Tensor values under 'qkv' [(heads + 2 kv_heads) D x H],
        'o' [H x heads D], 'gate', 'up' [I x H], 'down' [H x I]; cos_t, sin_t:
        the rotary tables of nvfp4_gemm_rope, as wide as half the rotated
        columns (a position past their last row is reported in the device
        status and rotated as that row).  q_norm, k_norm: bf16 [D], the norms of
        the query and key heads, or None; halves: the rotation pairs column i with
        column i + half of the rotated ones instead of 2i with 2i + 1.  expand: over
        a KVCache4, scratch["expanded"] are bf16 pages (3.6 times one layer's cache) where
        a request of the plan may have more rows than one pass over the codes takes:
        prompts, chunks, also one among decoding requests.  False: none, for plans whose
        requests have a few tokens each (a step of them is 5 us a layer faster then, and
        one with a chunk in it several times slower)."""
        self.plan, self.cache, self.w, self.eps = plan, cache, weights, eps
        self.attn_norm, self.mlp_norm, self.cos_t, self.sin_t = attn_norm, mlp_norm, cos_t, sin_t
        self.q_norm, self.k_norm, self.halves = q_norm, k_norm, halves
        T, H, I = plan.tokens, weights["o"].rows, weights["gate"].rows
        heads, kv_heads = plan.heads, plan.kv_heads
        N = weights["qkv"].rows
        self.head_dim = D = N // (heads + 2 * kv_heads)
        if N != (heads + 2 * kv_heads) * D or weights["o"].cols != heads * D:
            raise ValueError("qkv and o do not fit the plan's heads")
        if bool(plan.page_size) != (cache is not None):
            raise ValueError("a plan with pages goes with a cache, one without goes without")
        if cache is not None and (cache.page_size, cache.kv_heads, cache.head_dim) != (plan.page_size, kv_heads, D):
            raise ValueError(f"a cache of pages of {cache.page_size} tokens, {cache.kv_heads} heads of {cache.head_dim} "
                             f"columns does not fit a plan of {plan.page_size}, {kv_heads} and {D}")
        for name, norm in (("q_norm", q_norm), ("k_norm", k_norm)):
            if norm is not None and (norm.dtype != torch.bfloat16 or tuple(norm.shape) != (D,)):
                raise ValueError(f"{name} must be a bf16 [{D}] tensor")
        if halves and cos_t.shape[1] % 8:
            raise ValueError("halves: tables of a multiple of 8 columns")
        dev = attn_norm.device
        # prompts over a 4-bit cache: bf16 pages, taken out once per layer and step
        # (whether they are is nvfp4_attn_paged4's decision, from each step's lengths)
        self.four = isinstance(cache, KVCache4)
        self.expands = expands = self.four and expand and (T > plan.requests or heads // kv_heads > _PASS_ROWS)
        if scratch is None:
            scratch = {
                "h": NVFP4Tensor.empty(T, H, dev), "a": NVFP4Tensor.empty(T, heads * D, dev),
                "qkv": torch.empty((T, N), dtype=torch.bfloat16, device=dev),
                "attn": torch.empty((T, heads * D), dtype=torch.bfloat16, device=dev),
                "x1": torch.empty((T, H), dtype=torch.bfloat16, device=dev),
                "g_inter": torch.ones((1,), dtype=torch.float32, device=dev),
                "ws_amax": workspace(256, dev), "ws_gemm": workspace(gemm_workspace_bytes(), dev),
                "ws_attn": workspace(attn_workspace_bytes(), dev),
                "ws_mlp": workspace(mlp_workspace_bytes(T, H, I, NVFP4_INTER_DYNAMIC), dev),
                "expanded": KVCache.empty(cache.pages, kv_heads, cache.page_size, D, dev) if expands else None,
            }
        elif not (scratch["h"].rows == scratch["a"].rows == T and scratch["h"].cols == H and
                  scratch["a"].cols == heads * D and tuple(scratch["qkv"].shape) == (T, N) and
                  scratch["ws_mlp"].numel() >= mlp_workspace_bytes(T, H, I, NVFP4_INTER_DYNAMIC)):
            raise ValueError("scratch is a layer's of other sizes")
        elif expands and (scratch.get("expanded") is None or
                          scratch["expanded"].k.shape != (cache.pages, kv_heads, cache.page_size, D)):
            raise ValueError("scratch has no bf16 pages of the cache's sizes")
        self.scratch = scratch

    def forward(self, x: torch.Tensor, out: torch.Tensor, stream=None):
        """x, out: bf16 [T x H] (may alias), T the plan's tokens; after
        nvfp4_attn_plan of the step on the same stream.  Rows past the step's
        last token hold what their x gives."""
        s, plan, w = self.scratch, self.plan, self.w
        T, heads, kv_heads, D = plan.tokens, plan.heads, plan.kv_heads, self.head_dim
        if x.shape != s["x1"].shape or out.shape != x.shape:
            raise ValueError(f"x and out must be {tuple(s['x1'].shape)}, not {tuple(x.shape)} and {tuple(out.shape)}")
        nvfp4_scale_quantize(x, s["h"], s["ws_amax"], self.attn_norm, self.eps, stream)
        rows = s["qkv"].view(T, heads + 2 * kv_heads, D)
        q, k, v = rows[:, :heads], rows[:, heads:heads + kv_heads], rows[:, heads + kv_heads:]
        a = s["attn"].view(T, heads, D)
        cache = self.cache
        if self.q_norm is not None or self.k_norm is not None or self.halves:
            nvfp4_gemm(s["h"], w["qkv"], s["qkv"], None, stream, s["ws_gemm"])
            nvfp4_qk_norm_rope(q, k, self.q_norm, self.k_norm, plan.pos, self.cos_t, self.sin_t, halves=self.halves,
                               eps=self.eps, v=None if cache is None else v, plan=None if cache is None else plan,
                               cache=cache, stream=stream)
        else:
            nvfp4_gemm_rope(s["h"], w["qkv"], s["qkv"], plan.pos, self.cos_t, self.sin_t, 0, heads + kv_heads, D,
                            2 * self.cos_t.shape[1], False, stream, s["ws_gemm"])
            if cache is not None:
                (nvfp4_kv4_append if self.four else nvfp4_kv_append)(k, v, plan, cache, stream)
        # rows of padding count in the next quantization's scale: zero, so that
        # nothing of an earlier step is left in them
        if self.four:
            nvfp4_attn_paged4(q, cache, plan, a, s["ws_attn"], stream=stream, zero_padding=True,
                              expanded=s["expanded"] if self.expands else None)
        elif cache is not None:
            nvfp4_attn_paged(q, cache, plan, a, s["ws_attn"], stream=stream, zero_padding=True)
        else:
            nvfp4_attn_prompt(q, k, v, plan, a, s["ws_attn"], stream=stream, zero_padding=True)
        nvfp4_scale_quantize(s["attn"], s["a"], s["ws_amax"], None, self.eps, stream)
        nvfp4_gemm(s["a"], w["o"], s["x1"], x, stream, s["ws_gemm"])
        nvfp4_mlp(s["x1"], self.mlp_norm, w["gate"], w["up"], w["down"], NVFP4_INTER_DYNAMIC, s["g_inter"], out,
                  s["ws_mlp"], True, self.eps, stream)
