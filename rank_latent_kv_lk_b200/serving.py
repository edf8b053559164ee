"""Torch-facing wrappers of the serving operators (lk_serving.h): a paged
key-value cache with decode attention and eviction, products with 4-bit
weights, and the norms around a block.

Marshalling only.  What the C ABI cannot see -- a tensor's shape, strides,
type and device -- is checked here (ValueError, TypeError); the rest is the
library's (LkError).  Every call runs on its tensors' device and on that
device's current stream, or on `stream`; scratch memory comes from torch's
allocator per call, so calls on several streams and captured graphs share none.
"""
from __future__ import annotations

import ctypes as C
import math

import torch

from ._lib import LK_BF16, LK_F16, LK_F32, LK_I8, PagedCacheDesc, check, lib

_DT = {torch.float32: LK_F32, torch.bfloat16: LK_BF16, torch.float16: LK_F16, torch.int8: LK_I8}
_raw_stream = torch._C._cuda_getCurrentRawStream


def _code(dtype, allowed):
    if dtype not in allowed:
        raise TypeError(f"unsupported dtype {dtype}")
    return _DT[dtype]


def _elsewhere(device, stream):
    """Whether the call has to enter its tensors' device or the given stream first."""
    return stream is not None or device.index is None or device.index != torch.cuda.current_device()


def _enter(device, stream, fn, *args, **kw):
    """The call inside its device and stream."""
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, not {device}")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        return fn(*args, **kw)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _same(name, t, shape, dtype, device):
    """A contiguous tensor of this shape, type and device."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, not {dtype}")
    if t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor of shape {tuple(shape)} on {device} is needed, not "
                         f"{tuple(t.shape)} with strides {t.stride()} on {t.device}")


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

    def _set(self, k, v, k_scale, v_scale, mass, pos):
        _code(k.dtype, (torch.bfloat16, torch.float16, torch.int8))
        if k.dim() != 4 or k.device.type != "cuda":
            raise ValueError("k: a CUDA tensor [n_pages, n_kv_heads, page_size, head_dim] is needed")
        dev, rows = k.device, k.shape[:3]
        _same("k", k, k.shape, k.dtype, dev)
        _same("v", v, k.shape, k.dtype, dev)
        if (k.dtype is torch.int8) != (k_scale is not None) or (k_scale is None) != (v_scale is None):
            raise ValueError("k_scale and v_scale belong to an int8 cache, and only to it")
        if (mass is None) != (pos is None):
            raise ValueError("mass and pos come together")
        if k_scale is not None:
            _same("k_scale", k_scale, rows, torch.float32, dev)
            _same("v_scale", v_scale, rows, torch.float32, dev)
        if mass is not None:
            _same("mass", mass, rows, torch.float32, dev)
            _same("pos", pos, rows, torch.int32, dev)
        self.k, self.v, self.k_scale, self.v_scale, self.mass, self.pos = k, v, k_scale, v_scale, mass, pos
        self.device, self.dtype, self.rows = dev, k.dtype, rows
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self._desc = PagedCacheDesc(self.n_pages, self.page_size, self.n_kv_heads, self.head_dim, _DT[k.dtype],
                                    k.data_ptr(), v.data_ptr(), _ptr(k_scale), _ptr(v_scale), _ptr(mass), _ptr(pos))
        self._ref = C.byref(self._desc)

    def desc(self):
        return self._ref


def _table(cache, page_table, batch):
    if page_table.dim() != 2 or page_table.shape[0] != batch:
        raise ValueError(f"page_table: [{batch}, width] is needed, not {tuple(page_table.shape)}")
    _same("page_table", page_table, page_table.shape, torch.int32, cache.device)
    return page_table.shape[1]


def _new_tokens(cache, name, t):
    """Elements between the tokens of [batch, n_new, n_kv_heads, head_dim]."""
    if t.dim() != 4 or t.shape[2] != cache.n_kv_heads or t.shape[3] != cache.head_dim or t.device != cache.device:
        raise ValueError(f"{name}: [batch, n_new, {cache.n_kv_heads}, {cache.head_dim}] on {cache.device} is needed, "
                         f"not {tuple(t.shape)} on {t.device}")
    b, n, h, d = t.shape
    sb, sn, sh, sd = t.stride()
    step = sn if n > 1 else (sb if b > 1 else h * d)
    if sd != 1 or (h > 1 and sh != d) or (b > 1 and n > 1 and sb != n * step):
        raise ValueError(f"{name}: heads must be contiguous within a token and tokens evenly spaced, strides are "
                         f"{t.stride()}")
    return step


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
    if _elsewhere(cache.device, stream):
        return _enter(cache.device, stream, paged_append, cache, page_table, k_new, v_new, seq_len, next_pos, new_len,
                      seq_len_out, next_pos_out)
    step = _new_tokens(cache, "k_new", k_new)
    if v_new.shape != k_new.shape or v_new.dtype is not k_new.dtype or _new_tokens(cache, "v_new", v_new) != step:
        raise ValueError("k_new and v_new must have the same shape, type and token spacing")
    batch, n_new = k_new.shape[:2]
    width = _table(cache, page_table, batch)
    if seq_len_out is None:
        seq_len_out = seq_len
    if next_pos_out is None:
        next_pos_out = next_pos
    for name, t in (("seq_len", seq_len), ("seq_len_out", seq_len_out), ("next_pos", next_pos),
                    ("next_pos_out", next_pos_out), ("new_len", new_len)):
        if t is not None:
            _same(name, t, (batch,), torch.int32, cache.device)
    check(lib.lk_paged_append(cache._ref, page_table.data_ptr(), batch, width, k_new.data_ptr(), v_new.data_ptr(),
                              _code(k_new.dtype, (torch.bfloat16, torch.float16)), step, n_new, _ptr(new_len),
                              seq_len.data_ptr(), seq_len_out.data_ptr(), _ptr(next_pos), _ptr(next_pos_out),
                              _raw_stream(cache.device.index)))


def paged_decode_attn(cache, page_table, q, seq_len, max_seq_len, softmax_scale=None, accumulate=False, out=None,
                      out_dtype=None, stream=None):
    """softmax(q K^T * scale) V of one new token per sequence over its pages.

    q: [batch, n_heads, head_dim], heads contiguous within a sequence, n_heads a
    multiple of the cache's kv heads; seq_len: device int32 [batch];
    max_seq_len: host bound.  accumulate: add every cached token's attention
    weight, summed over the heads of its group, to cache.mass.
    """
    if _elsewhere(cache.device, stream):
        return _enter(cache.device, stream, paged_decode_attn, cache, page_table, q, seq_len, max_seq_len,
                      softmax_scale, accumulate, out, out_dtype)
    if q.dim() != 3 or q.shape[2] != cache.head_dim or q.device != cache.device:
        raise ValueError(f"q: [batch, n_heads, {cache.head_dim}] on {cache.device} is needed, not {tuple(q.shape)} "
                         f"on {q.device}")
    batch, heads, dim = q.shape
    qs = q.stride()
    if qs[2] != 1 or (heads > 1 and qs[1] != dim):
        raise ValueError(f"q: heads must be contiguous within a sequence, strides are {qs}")
    width = _table(cache, page_table, batch)
    _same("seq_len", seq_len, (batch,), torch.int32, cache.device)
    if out is None:
        out = torch.empty((batch, heads, dim), dtype=out_dtype or q.dtype, device=cache.device)
    else:
        _same("out", out, q.shape, out.dtype, cache.device)
    acc = 1 if accumulate else 0
    need = lib.lk_paged_decode_workspace_bytes(cache._ref, batch, heads, max_seq_len, acc)
    ws = torch.empty(need, dtype=torch.uint8, device=cache.device)
    check(lib.lk_paged_decode_attn(
        cache._ref, page_table.data_ptr(), batch, width, q.data_ptr(),
        _code(q.dtype, (torch.bfloat16, torch.float16)), heads, qs[0] if batch > 1 else heads * dim,
        seq_len.data_ptr(), max_seq_len, 1.0 / math.sqrt(dim) if softmax_scale is None else softmax_scale, acc,
        out.data_ptr(), _code(out.dtype, (torch.bfloat16, torch.float16, torch.float32)), ws.data_ptr(), need,
        _raw_stream(cache.device.index)))
    return out


def paged_evict(cache, page_table, seq_len, next_pos, max_seq_len, budget, window=0, n_sink=0, mass_out=None,
                pos_out=None, seq_len_out=None, stream=None):
    """Cut every sequence longer than `budget` to its most wanted tokens, per kv head.

    Kept first: tokens at positions below n_sink or among the last `window`
    (from next_pos), then the largest accumulated weight, then the lowest slot.
    Kept tokens behind the budget move into the free slots below it.  The kept
    rows' mass and positions go to mass_out / pos_out and the lengths to
    seq_len_out (default: in place).
    """
    if _elsewhere(cache.device, stream):
        return _enter(cache.device, stream, paged_evict, cache, page_table, seq_len, next_pos, max_seq_len, budget,
                      window, n_sink, mass_out, pos_out, seq_len_out)
    if cache.mass is None:
        raise ValueError("eviction needs a cache with mass and pos")
    if mass_out is None:
        mass_out = cache.mass
    if pos_out is None:
        pos_out = cache.pos
    if seq_len_out is None:
        seq_len_out = seq_len
    if seq_len.dim() != 1:
        raise ValueError("seq_len: [batch] is needed")
    batch = seq_len.shape[0]
    width = _table(cache, page_table, batch)
    for name, t in (("seq_len", seq_len), ("next_pos", next_pos), ("seq_len_out", seq_len_out)):
        _same(name, t, (batch,), torch.int32, cache.device)
    _same("mass_out", mass_out, cache.rows, torch.float32, cache.device)
    _same("pos_out", pos_out, cache.rows, torch.int32, cache.device)
    need = lib.lk_paged_evict_workspace_bytes(cache._ref, batch, max_seq_len, budget)
    ws = torch.empty(need, dtype=torch.uint8, device=cache.device)
    check(lib.lk_paged_evict(cache._ref, page_table.data_ptr(), batch, width, seq_len.data_ptr(), next_pos.data_ptr(),
                             max_seq_len, budget, window, n_sink, mass_out.data_ptr(), pos_out.data_ptr(),
                             seq_len_out.data_ptr(), ws.data_ptr(), need, _raw_stream(cache.device.index)))


class W4Weight:
    """4-bit weight [n_out, k_in] laid out for w4_linear: codes uint8 [n_out,
    k_in / 2] (two's-complement nibbles, low nibble = even input), scales fp16
    [n_out, k_in / group], group 32, 64 or 128.  With up_codes and up_scales of
    the same sizes the product is silu(x gate^T) * (x up^T)."""

    def __init__(self, codes, scales, up_codes=None, up_scales=None):
        dev = codes.device
        if codes.dim() != 2 or scales.dim() != 2 or dev.type != "cuda" or scales.shape[1] < 1:
            raise ValueError("codes and scales must be CUDA matrices")
        self.n_out, self.k_in = codes.shape[0], 2 * codes.shape[1]
        self.group = self.k_in // scales.shape[1]
        if self.group * scales.shape[1] != self.k_in:
            raise ValueError(f"{scales.shape[1]} scale groups do not divide {self.k_in} inputs")
        if (up_codes is None) != (up_scales is None):
            raise ValueError("up_codes and up_scales come together")
        self.gated, self.device = up_codes is not None, dev
        for name, c, s in (("", codes, scales), ("up_", up_codes, up_scales)):
            if c is not None:
                _same(name + "codes", c, codes.shape, torch.uint8, dev)
                _same(name + "scales", s, (self.n_out, scales.shape[1]), torch.float16, dev)
        with torch.cuda.device(dev):
            need = lib.lk_w4_packed_bytes(self.n_out, self.k_in, self.group, int(self.gated))
            self.packed = torch.empty(need, dtype=torch.uint8, device=dev)
            check(lib.lk_w4_pack(codes.data_ptr(), scales.data_ptr(), _ptr(up_codes), _ptr(up_scales), self.n_out,
                                 self.k_in, self.group, self.packed.data_ptr(), need, _raw_stream(dev.index)))


def w4_linear(w, x, residual=None, y=None, y_dtype=None, stream=None):
    """x W^T (+ residual), or silu(x gate^T) * (x up^T) for a gated weight.

    x: [m, k_in] bf16 or fp16, rows contiguous; residual: [m, n_out] of x's type.
    """
    if _elsewhere(w.device, stream):
        return _enter(w.device, stream, w4_linear, w, x, residual, y, y_dtype)
    if x.dim() != 2 or x.shape[1] != w.k_in or x.stride(1) != 1 or x.device != w.device:
        raise ValueError(f"x: [m, {w.k_in}] with contiguous rows on {w.device} is needed, not {tuple(x.shape)} with "
                         f"strides {x.stride()} on {x.device}")
    m = x.shape[0]
    if y is None:
        y = torch.empty((m, w.n_out), dtype=y_dtype or x.dtype, device=w.device)
    else:
        _same("y", y, (m, w.n_out), y.dtype, w.device)
    if residual is not None:
        _same("residual", residual, (m, w.n_out), x.dtype, w.device)
    check(lib.lk_w4_linear(w.packed.data_ptr(), w.n_out, w.k_in, w.group, 1 if w.gated else 0, x.data_ptr(),
                           _code(x.dtype, (torch.bfloat16, torch.float16)), m, x.stride(0) if m > 1 else w.k_in,
                           _ptr(residual), y.data_ptr(), _code(y.dtype, (torch.bfloat16, torch.float16, torch.float32)),
                           _raw_stream(w.device.index)))
    return y


def rmsnorm_gate_residual(y, x, w_post=None, gate=None, scale=1.0, w_pre=None, eps=1e-5, x_out=None, h=None,
                          stream=None):
    """x + scale * gate * (RMSNorm(y) * w_post), and RMSNorm of that * w_pre.

    y, x: [m, width]; w_post, w_pre: [width] (w_post None: y enters as it is;
    w_pre None: no second norm); gate: [width] or [m, width].  x_out may be x or
    y and h may be y.  Returns (x_out, h); h is None without w_pre.
    """
    dev = y.device
    if _elsewhere(dev, stream):
        return _enter(dev, stream, rmsnorm_gate_residual, y, x, w_post, gate, scale, w_pre, eps, x_out, h)
    dtype = y.dtype
    code = _code(dtype, (torch.float32, torch.bfloat16, torch.float16))
    if y.dim() != 2:
        raise ValueError("y: [m, width] is needed")
    shape = y.shape
    m, width = shape
    _same("y", y, shape, dtype, dev)
    _same("x", x, shape, dtype, dev)
    if w_post is not None:
        _same("w_post", w_post, (width,), dtype, dev)
    per_row = 0
    if gate is not None:
        per_row = 1 if gate.dim() == 2 else 0
        _same("gate", gate, shape if per_row else (width,), dtype, dev)
    if x_out is None:
        x_out = torch.empty_like(x)
    else:
        _same("x_out", x_out, shape, dtype, dev)
    if w_pre is not None:
        _same("w_pre", w_pre, (width,), dtype, dev)
        if h is None:
            h = torch.empty_like(x)
        else:
            _same("h", h, shape, dtype, dev)
    elif h is not None:
        raise ValueError("h needs w_pre")
    if m == 0:
        return x_out, h
    check(lib.lk_rmsnorm_gate_residual(y.data_ptr(), x.data_ptr(), _ptr(w_post), _ptr(gate), per_row, _ptr(w_pre),
                                       code, m, width, scale, eps, x_out.data_ptr(), _ptr(h), _raw_stream(dev.index)))
    return x_out, h
