"""One W8A8 pre-norm decoder layer with latent attention and LASER hybrid FFN.

Composition (the pages do not describe the block; a LLaMA-style pre-norm
layer with unit RMSNorm weights, eps 1e-5, no positional rotation):

  x_q      = int8(RMSNorm(x))
  q        = x_q W_Q^T                      (W8A8 dense linear)
  latents  = quant(x_q A^T) appended        (lk_latent_decode_step: append,
  a        = latent attention                 then attention)
  x2       = x + int8(a) W_O^T              (W8A8 dense linear + residual)
  h_q      = int8(RMSNorm(x2))
  g, u     = hybrid(h_q; gate), hybrid(h_q; up)     (LASER hybrid linear)
  m_q      = int8(silu(g) * u)
  out      = x2 + hybrid(m_q; down)

Every step is a call into the C ABI; this module only wires buffers.

W4PagedDecoderLayer is its neighbour for layers whose K and V stay dense: 4-bit
weights, grouped heads over a paged key-value cache, eviction by accumulated
attention weight, and the norms around a block fused with its residual.
"""
from __future__ import annotations

import torch

from .api import (LatentCache, LowrankWeight, latent_decode_step, lowrank_linear, quantize_rows_i8,
                  rmsnorm_quant_i8, swiglu_quant_i8)


def dense_weight(W, s, device):
    """A plain W8A8 linear as a hybrid linear whose every input channel is dense."""
    n_out, k_in = W.shape
    idx = torch.arange(k_in, dtype=torch.int32, device=device)
    return LowrankWeight(k_in, n_out, 0, idx, None, W.to(device), s.to(device), None, None, None, None)


def hybrid_weight(d, k_in, n_out, device):
    t = {k: v.to(device) for k, v in d.items()}
    return LowrankWeight(k_in, n_out, int(t["U"].shape[0]), t["dense_idx"], t["lr_idx"], t["W_D"], t["s_D"],
                         t["U"], t["s_U"], t["V"], t["s_V"])


class W8A8DecoderLayer:
    def __init__(self, weights, n_heads, head_dim, ranks_k, ranks_v, batch, capacity, ffn_inter,
                 device="cuda"):
        E = weights["W_Q"].shape[1]
        self.E, self.n_heads, self.head_dim = E, n_heads, head_dim
        self.batch = batch
        self.wq = dense_weight(weights["W_Q"], weights["s_Q"], device)
        self.wo = dense_weight(weights["W_O"], weights["s_O"], device)
        self.A = weights["A"].to(device)
        self.s_A = weights["s_A"].to(device)
        self.B_K = weights["B_K"].to(device)
        self.B_V = weights["B_V"].to(device)
        self.gate = hybrid_weight(weights["gate"], E, ffn_inter, device)
        self.up = hybrid_weight(weights["up"], E, ffn_inter, device)
        self.down = hybrid_weight(weights["down"], ffn_inter, E, device)
        self.cache_k = LatentCache(batch, ranks_k, capacity, "i8", 32, device)
        self.cache_v = LatentCache(batch, ranks_v, capacity, "i8", 32, device, role="v")

    def step(self, x, seq_len, lens, trace=None):
        """x: [B, E] bf16 (device); seq_len: device int32 [B]; lens: host list (advanced in place).

        If `trace` is a dict, the intermediate device tensors are stored in it."""
        B = x.shape[0]
        xq, sx = rmsnorm_quant_i8(x)
        q = lowrank_linear(self.wq, xq, sx)
        # append the new token's latents, then attend (the attention launch
        # overlaps the append)
        attn = latent_decode_step(self.cache_k, self.cache_v, xq, self.A, seq_len, lens,
                                  q.view(B, self.n_heads, self.head_dim), self.B_K, self.B_V, x_scale=sx,
                                  a_scale=self.s_A, out_dtype=torch.bfloat16)
        for b in range(B):
            lens[b] += 1
        aq, sa = quantize_rows_i8(attn.view(B, self.n_heads * self.head_dim))
        x2 = lowrank_linear(self.wo, aq, sa, residual=x)
        hq, sh = rmsnorm_quant_i8(x2)
        g = lowrank_linear(self.gate, hq, sh)
        u = lowrank_linear(self.up, hq, sh)
        mq, sm = swiglu_quant_i8(g, u)
        out = lowrank_linear(self.down, mq, sm, residual=x2)
        if trace is not None:
            trace.update(xq=xq, sx=sx, q=q, attn=attn, aq=aq, sa=sa, x2=x2, hq=hq, sh=sh, gate=g, up=u, mq=mq,
                         sm=sm, out=out)
        return out


class W4PagedDecoderLayer:
    """One pre-norm decoder layer with 4-bit weights and a paged K/V cache.

    step(): h is the normed input (the previous layer's second result, or
    rmsnorm_gate_residual of the embedding), x the residual stream:

      q, k, v  = h W_QKV^T                     (4-bit; k, v appended to the pages)
      a        = attention over the pages      (weights accumulated if the cache has mass)
      x, h     = x + g_1 . post_1(a W_O^T),  RMSNorm . w_ffn
      m        = silu(h W_gate^T) * (h W_up^T) (4-bit, one launch)
      x, h     = x + g_2 . post_2(m W_down^T), RMSNorm . w_next

    weights: (codes, scales) for "qkv" [(n_heads + 2 n_kv_heads) head_dim, E],
    "o", "gate", "up", "down" (codes and scales as W4Weight); [E] tensors
    "norm_ffn", "norm_next" and optionally "post_attn", "post_ffn" (norms
    behind a block) and "gate_attn", "gate_ffn" (its gate).
    """

    def __init__(self, weights, n_heads, n_kv_heads, head_dim, n_pages, page_size, cache_dtype=torch.bfloat16,
                 mass=False, eps=1e-5, device="cuda"):
        # here and not above: W8A8DecoderLayer does without the serving operators' binding
        from . import serving
        self._op = serving
        self.n_heads, self.n_kv_heads, self.head_dim, self.eps = n_heads, n_kv_heads, head_dim, eps

        def w4(*names):
            return serving.W4Weight(*[t.to(device) for n in names for t in weights[n]])

        self.qkv, self.o, self.gate_up, self.down = w4("qkv"), w4("o"), w4("gate", "up"), w4("down")
        self.norm = {k: None if weights.get(k) is None else weights[k].to(device)
                     for k in ("norm_ffn", "norm_next", "post_attn", "post_ffn", "gate_attn", "gate_ffn")}
        self.cache = serving.PagedKVCache(n_pages, page_size, n_kv_heads, head_dim, cache_dtype, mass, device)

    def step(self, x, h, page_table, seq_len, max_seq_len, next_pos=None):
        """x, h: [B, E]; page_table, seq_len, next_pos: device int32 (lengths and positions advance by one in
        place); max_seq_len: host bound on the lengths after the step."""
        B, nh, nk, D, n, op = x.shape[0], self.n_heads, self.n_kv_heads, self.head_dim, self.norm, self._op
        qkv = op.w4_linear(self.qkv, h)
        q = qkv[:, :nh * D].view(B, nh, D)
        k = qkv[:, nh * D:(nh + nk) * D].view(B, 1, nk, D)
        v = qkv[:, (nh + nk) * D:].view(B, 1, nk, D)
        op.paged_append(self.cache, page_table, k, v, seq_len, next_pos)
        a = op.paged_decode_attn(self.cache, page_table, q, seq_len, max_seq_len,
                                 accumulate=self.cache.mass is not None)
        y = op.w4_linear(self.o, a.view(B, nh * D))
        x, h = op.rmsnorm_gate_residual(y, x, n["post_attn"], n["gate_attn"], 1.0, n["norm_ffn"], self.eps)
        y = op.w4_linear(self.down, op.w4_linear(self.gate_up, h))
        return op.rmsnorm_gate_residual(y, x, n["post_ffn"], n["gate_ffn"], 1.0, n["norm_next"], self.eps)

    def evict(self, page_table, seq_len, next_pos, max_seq_len, budget, window=0, n_sink=0):
        """Cut the sequences to `budget` cached tokens per kv head (lengths in place)."""
        self._op.paged_evict(self.cache, page_table, seq_len, next_pos, max_seq_len, budget, window, n_sink)
