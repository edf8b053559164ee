"""Torch-facing wrappers of the serving operators (lk_serving.h): a paged
key-value cache with decode attention and eviction, products with 4-bit
weights, and the norms around a block.

The checks of shapes, strides, types and devices (ValueError, TypeError) and
the calls stand in the binding (csrc/lk_serving_py.cpp); what the library
refuses raises LkError.  Every call runs on its tensors' device and on that
device's current stream, or on `stream`.  Outputs and scratch memory come from
torch's allocator per call, so calls on several streams and captured graphs
share none.  No sequences or rows at all are no error: nothing is done.

A call on `stream` is ordered with nothing else: the caller makes that stream
wait for the inputs (stream.wait_stream) and waits for it before using the
result.  Both may be freed without waiting.
"""
from __future__ import annotations

import torch

from . import _lib  # noqa: F401  (fails loudly if the library is missing)
from . import _serving_ext as _ext


def _on(stream, device, fn, *args):
    """The call with `stream` current, which has to be the tensors' device's.  The memory of the inputs, which another
    stream's pool may own, is not given out again before the call is done, nor the result's before the caller's stream
    is done with it."""
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    caller = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        out = fn(*args)
    if stream != caller:
        for a in args:
            for t in _tensors_of(a):
                t.record_stream(stream)
        for t in out if isinstance(out, tuple) else (out,):
            if t is not None:
                t.record_stream(caller)
    return out


def _tensors_of(a):
    if isinstance(a, torch.Tensor):
        return (a,)
    if isinstance(a, PagedKVCache):
        return tuple(t for t in (getattr(a, n) for n in _TENSORS) if t is not None)
    return (a.packed,) if isinstance(a, W4Weight) else ()


_TENSORS = ("k", "v", "k_scale", "v_scale", "mass", "pos")


def _tensor(name):
    """A tensor of a PagedKVCache: assigning one replaces it for every later call."""
    def get(self):
        return getattr(self._c, name)

    def put(self, t):
        self._set(*[t if n == name else getattr(self._c, n) for n in _TENSORS])

    return property(get, put)


def _size(i):
    return property(lambda self: self._c.k.shape[i])


class PagedKVCache:
    """Paged K and V of one layer: pages of `page_size` rows per kv head.

    k, v: [n_pages, n_kv_heads, page_size, head_dim] bf16, fp16 or int8 (with
    fp32 scales [n_pages, n_kv_heads, page_size]).  mass / pos, of the scales'
    shape: accumulated attention weight and position of every row, for a cache
    that is evicted from.  Which pages a sequence has is the caller's page
    table, int32 [batch, width] on the device.
    """

    def __init__(self, n_pages, page_size, n_kv_heads, head_dim, dtype=torch.bfloat16, mass=False, device="cuda"):
        shape = (n_pages, n_kv_heads, page_size, head_dim)

        def rows(t):
            return torch.zeros(shape[:3], dtype=t, device=device)

        i8 = dtype is torch.int8
        self._set(torch.zeros(shape, dtype=dtype, device=device), torch.zeros(shape, dtype=dtype, device=device),
                  rows(torch.float32) if i8 else None, rows(torch.float32) if i8 else None,
                  rows(torch.float32) if mass else None, rows(torch.int32) if mass else None)

    @classmethod
    def from_tensors(cls, k, v, k_scale=None, v_scale=None, mass=None, pos=None):
        """A cache over the caller's tensors (kept alive, not copied)."""
        self = cls.__new__(cls)
        self._set(k, v, k_scale, v_scale, mass, pos)
        return self

    def _set(self, *tensors):
        self._c = _ext.PagedCache(*tensors)  # refuses tensors that do not fit together

    # The binding's own tensors, so that what is shown here is what the calls use.
    k, v, k_scale, v_scale, mass, pos = (_tensor(n) for n in _TENSORS)
    device = property(lambda self: self._c.k.device)
    dtype = property(lambda self: self._c.k.dtype)
    n_pages, n_kv_heads, page_size, head_dim = (_size(i) for i in range(4))


def paged_append(cache, page_table, k_new, v_new, seq_len, next_pos=None, new_len=None, seq_len_out=None,
                 next_pos_out=None, stream=None):
    """Append new tokens to every sequence's pages and advance its length.

    k_new, v_new: [batch, n_new, n_kv_heads, head_dim], heads contiguous within
    a token (views of one projection's output will do); int8 caches quantise
    each row.  seq_len: device int32 [batch]; new_len (int32 [batch], optional):
    how many of the n_new tokens each sequence takes.  A cache with mass needs
    next_pos, the position of each sequence's next token.  The new lengths and
    positions go to seq_len_out / next_pos_out (default: in place).
    """
    if stream is not None:
        return _on(stream, cache.device, paged_append, cache, page_table, k_new, v_new, seq_len, next_pos, new_len,
                   seq_len_out, next_pos_out)
    _ext.paged_append(cache._c, page_table, k_new, v_new, seq_len, next_pos, new_len, seq_len_out, next_pos_out)


def paged_decode_attn(cache, page_table, q, seq_len, max_seq_len, softmax_scale=None, accumulate=False, out=None,
                      out_dtype=None, stream=None):
    """softmax(q K^T * scale) V of one new token per sequence over its pages.

    q: [batch, n_heads, head_dim], heads contiguous within a sequence, n_heads a
    multiple of the cache's kv heads; seq_len: device int32 [batch];
    max_seq_len: host bound.  accumulate: add every cached token's attention
    weight, summed over the heads of its group, to cache.mass.  out: where the
    result goes, in its own type; without it, a new tensor of out_dtype
    (default: q's).
    """
    if stream is not None:
        return _on(stream, cache.device, paged_decode_attn, cache, page_table, q, seq_len, max_seq_len, softmax_scale,
                   accumulate, out, out_dtype)
    return _ext.paged_decode_attn(cache._c, page_table, q, seq_len, max_seq_len, softmax_scale, accumulate, out,
                                  out_dtype)


def paged_evict(cache, page_table, seq_len, next_pos, max_seq_len, budget, window=0, n_sink=0, mass_out=None,
                pos_out=None, seq_len_out=None, stream=None):
    """Cut every sequence longer than `budget` to its most wanted tokens, per kv head.

    Kept first: tokens at positions below n_sink or among the last `window`
    (from next_pos), then the largest accumulated weight, then the lowest slot.
    Kept tokens behind the budget move into the free slots below it.  The kept
    rows' mass and positions go to mass_out / pos_out and the lengths to
    seq_len_out (default: in place).
    """
    if stream is not None:
        return _on(stream, cache.device, paged_evict, cache, page_table, seq_len, next_pos, max_seq_len, budget, window,
                   n_sink, mass_out, pos_out, seq_len_out)
    _ext.paged_evict(cache._c, page_table, seq_len, next_pos, max_seq_len, budget, window, n_sink, mass_out, pos_out,
                     seq_len_out)


def _shown(name):
    return property(lambda self: getattr(self._c, name))


class W4Weight:
    """4-bit weight [n_out, k_in] laid out for w4_linear: codes uint8 [n_out,
    k_in / 2] (two's-complement nibbles, low nibble = even input), scales fp16
    [n_out, k_in / group], group 32, 64 or 128.  With up_codes and up_scales of
    the same sizes the product is silu(x gate^T) * (x up^T)."""

    def __init__(self, codes, scales, up_codes=None, up_scales=None):
        self._c = _ext.W4(codes, scales, up_codes, up_scales)

    packed, n_out, k_in, group, gated = (_shown(n) for n in ("packed", "n_out", "k_in", "group", "gated"))


def w4_linear(w, x, residual=None, y=None, y_dtype=None, stream=None):
    """x W^T (+ residual), or silu(x gate^T) * (x up^T) for a gated weight.

    x: [m, k_in] bf16 or fp16, rows contiguous; residual: [m, n_out] of x's type.
    y: where the result goes, in its own type; without it, a new tensor of
    y_dtype (default: x's).
    """
    if stream is not None:
        return _on(stream, w.packed.device, w4_linear, w, x, residual, y, y_dtype)
    return _ext.w4_linear(w._c, x, residual, y, y_dtype)


def rmsnorm_gate_residual(y, x, w_post=None, gate=None, scale=1.0, w_pre=None, eps=1e-5, x_out=None, h=None,
                          stream=None):
    """x + scale * gate * (RMSNorm(y) * w_post), and RMSNorm of that * w_pre.

    y, x: [m, width]; w_post, w_pre: [width] (w_post None: y enters as it is;
    w_pre None: no second norm); gate: [width] or [m, width].  x_out may be x or
    y and h may be y.  Returns (x_out, h); h is None without w_pre.
    """
    if stream is not None:
        return _on(stream, y.device, rmsnorm_gate_residual, y, x, w_post, gate, scale, w_pre, eps, x_out, h)
    return _ext.rmsnorm_gate_residual(y, x, w_post, gate, scale, w_pre, eps, x_out, h)
