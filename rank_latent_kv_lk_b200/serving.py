"""Torch-facing wrappers of the serving operators (lk_serving.h): a paged
key-value cache with decode attention and eviction, products with 4-bit
weights, and the norms around a block.

Marshalling only.  What the C ABI cannot see -- a tensor's shape, strides,
type and device -- is checked here (ValueError, TypeError); the rest is the
library's (LkError).  Every call runs on its tensors' device and on that
device's current stream, or on `stream`.  Scratch memory is kept per host
thread and stream, whose calls run one after another; a call that is captured
into a graph gets its own, from the graph's pool, so replays share none.
"""
from __future__ import annotations

import ctypes as C
import math
import threading

import torch

from ._lib import LK_BF16, LK_F16, LK_F32, LK_I8, PagedCacheDesc, check, lib

_DT = {torch.float32: LK_F32, torch.bfloat16: LK_BF16, torch.float16: LK_F16, torch.int8: LK_I8}
_FLOAT = {torch.float32: LK_F32, torch.bfloat16: LK_BF16, torch.float16: LK_F16}
_HALF = {torch.bfloat16: LK_BF16, torch.float16: LK_F16}
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_capturing = torch._C._cuda_isCurrentStreamCapturing
_i32 = torch.int32


def _code(dtype, allowed):
    try:
        return allowed[dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {dtype}") from None


class _Scratch(threading.local):
    """Scratch buffers of this thread's calls, one per stream."""

    def __init__(self):
        self.buffers = {}

    def get(self, index, stream, nbytes):
        if _capturing():
            return torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", index))
        buf = self.buffers.get((index, stream))
        if buf is None or buf.numel() < nbytes:
            # twice what is asked for, so that a growing cache reallocates seldom
            buf = torch.empty(2 * nbytes, dtype=torch.uint8, device=torch.device("cuda", index))
            self.buffers[index, stream] = buf
        return buf


_scratch = _Scratch()


def _enter(device, stream, fn, *args):
    """The call inside its tensors' device and the given stream."""
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, not {device}")
    if stream is not None and stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        return fn(*args)


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
        _code(k.dtype, _DT)
        if k.dtype is torch.float32:
            raise TypeError("a paged cache holds bf16, fp16 or int8")
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
        self.device, self.dtype, self.rows, self.index = dev, k.dtype, rows, dev.index
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self._desc = PagedCacheDesc(self.n_pages, self.page_size, self.n_kv_heads, self.head_dim, _DT[k.dtype],
                                    k.data_ptr(), v.data_ptr(), _ptr(k_scale), _ptr(v_scale), _ptr(mass), _ptr(pos))
        self._ref = C.byref(self._desc)
        self._scale = 1.0 / math.sqrt(self.head_dim)
        self._need = {}

    def desc(self):
        return self._ref

    def _decode_bytes(self, batch, heads, max_len, acc):
        """Workspace of a decode call, asked for once per 1024 tokens of the bound (it grows with it)."""
        key = (batch, heads, (max_len + 1023) >> 10, acc)
        need = self._need.get(key)
        if need is None:
            need = (lib.lk_paged_decode_workspace_bytes(self._ref, batch, heads, key[2] << 10, acc) or
                    lib.lk_paged_decode_workspace_bytes(self._ref, batch, heads, max_len, acc))
            if need:
                self._need[key] = need
        return need


def _table(cache, page_table, batch):
    """The page table's width."""
    shape = page_table.shape
    if len(shape) != 2 or shape[0] != batch or page_table.dtype is not _i32 or not page_table.is_contiguous() \
            or page_table.get_device() != cache.index:
        raise ValueError(f"page_table: a contiguous int32 [{batch}, width] on {cache.device} is needed, not "
                         f"{page_table.dtype} {tuple(shape)} on {page_table.device}")
    return shape[1]


def _counts(name, t, batch, cache):
    """An int32 vector of the batch."""
    if t.dtype is not _i32 or t.shape != (batch,) or not t.is_contiguous() or t.get_device() != cache.index:
        raise ValueError(f"{name}: a contiguous int32 [{batch}] on {cache.device} is needed, not {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")


def _new_tokens(cache, name, t):
    """Elements between the tokens of [batch, n_new, n_kv_heads, head_dim]."""
    shape = t.shape
    if len(shape) != 4 or shape[2] != cache.n_kv_heads or shape[3] != cache.head_dim or t.get_device() != cache.index:
        raise ValueError(f"{name}: [batch, n_new, {cache.n_kv_heads}, {cache.head_dim}] on {cache.device} is needed, "
                         f"not {tuple(shape)} on {t.device}")
    b, n, h, d = shape
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
    if stream is not None or cache.index != _current_device():
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
            _counts(name, t, batch, cache)
    status = lib.lk_paged_append(cache._ref, page_table.data_ptr(), batch, width, k_new.data_ptr(), v_new.data_ptr(),
                                 _code(k_new.dtype, _HALF), step, n_new, _ptr(new_len), seq_len.data_ptr(),
                                 seq_len_out.data_ptr(), _ptr(next_pos), _ptr(next_pos_out), _raw_stream(cache.index))
    if status:
        check(status)


def paged_decode_attn(cache, page_table, q, seq_len, max_seq_len, softmax_scale=None, accumulate=False, out=None,
                      out_dtype=None, stream=None):
    """softmax(q K^T * scale) V of one new token per sequence over its pages.

    q: [batch, n_heads, head_dim], heads contiguous within a sequence, n_heads a
    multiple of the cache's kv heads; seq_len: device int32 [batch];
    max_seq_len: host bound.  accumulate: add every cached token's attention
    weight, summed over the heads of its group, to cache.mass.
    """
    if stream is not None or cache.index != _current_device():
        return _enter(cache.device, stream, paged_decode_attn, cache, page_table, q, seq_len, max_seq_len,
                      softmax_scale, accumulate, out, out_dtype)
    shape = q.shape
    if len(shape) != 3 or shape[2] != cache.head_dim or q.get_device() != cache.index:
        raise ValueError(f"q: [batch, n_heads, {cache.head_dim}] on {cache.device} is needed, not {tuple(shape)} "
                         f"on {q.device}")
    batch, heads, dim = shape
    step, inner, one = q.stride()
    if one != 1 or (heads > 1 and inner != dim):
        raise ValueError(f"q: heads must be contiguous within a sequence, strides are {q.stride()}")
    width = _table(cache, page_table, batch)
    _counts("seq_len", seq_len, batch, cache)
    if out is None:
        out = q.new_empty((batch, heads, dim)) if out_dtype is None else q.new_empty((batch, heads, dim), dtype=out_dtype)
    else:
        _same("out", out, shape, out.dtype, cache.device)
    acc = 1 if accumulate else 0
    need = cache._decode_bytes(batch, heads, max_seq_len, acc)
    raw = _raw_stream(cache.index)
    status = lib.lk_paged_decode_attn(
        cache._ref, page_table.data_ptr(), batch, width, q.data_ptr(), _code(q.dtype, _HALF), heads,
        step if batch > 1 else heads * dim, seq_len.data_ptr(), max_seq_len,
        cache._scale if softmax_scale is None else softmax_scale, acc, out.data_ptr(), _code(out.dtype, _FLOAT),
        _scratch.get(cache.index, raw, need).data_ptr(), need, raw)
    if status:
        check(status)
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
    if stream is not None or cache.index != _current_device():
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
        _counts(name, t, batch, cache)
    if mass_out is not cache.mass:
        _same("mass_out", mass_out, cache.rows, torch.float32, cache.device)
    if pos_out is not cache.pos:
        _same("pos_out", pos_out, cache.rows, torch.int32, cache.device)
    need = lib.lk_paged_evict_workspace_bytes(cache._ref, batch, max_seq_len, budget)
    raw = _raw_stream(cache.index)
    status = lib.lk_paged_evict(cache._ref, page_table.data_ptr(), batch, width, seq_len.data_ptr(),
                                next_pos.data_ptr(), max_seq_len, budget, window, n_sink, mass_out.data_ptr(),
                                pos_out.data_ptr(), seq_len_out.data_ptr(),
                                _scratch.get(cache.index, raw, need).data_ptr(), need, raw)
    if status:
        check(status)


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
        self.gated, self.device, self.index = up_codes is not None, dev, dev.index
        for name, c, s in (("", codes, scales), ("up_", up_codes, up_scales)):
            if c is not None:
                _same(name + "codes", c, codes.shape, torch.uint8, dev)
                _same(name + "scales", s, (self.n_out, scales.shape[1]), torch.float16, dev)
        with torch.cuda.device(dev):
            need = lib.lk_w4_packed_bytes(self.n_out, self.k_in, self.group, int(self.gated))
            self.packed = torch.empty(need, dtype=torch.uint8, device=dev)
            self.packed_ptr = self.packed.data_ptr()
            check(lib.lk_w4_pack(codes.data_ptr(), scales.data_ptr(), _ptr(up_codes), _ptr(up_scales), self.n_out,
                                 self.k_in, self.group, self.packed_ptr, need, _raw_stream(dev.index)))


def w4_linear(w, x, residual=None, y=None, y_dtype=None, stream=None):
    """x W^T (+ residual), or silu(x gate^T) * (x up^T) for a gated weight.

    x: [m, k_in] bf16 or fp16, rows contiguous; residual: [m, n_out] of x's type.
    """
    if stream is not None or w.index != _current_device():
        return _enter(w.device, stream, w4_linear, w, x, residual, y, y_dtype)
    shape = x.shape
    if len(shape) != 2 or shape[1] != w.k_in or x.get_device() != w.index or x.stride(1) != 1:
        raise ValueError(f"x: [m, {w.k_in}] with contiguous rows on {w.device} is needed, not {tuple(shape)} with "
                         f"strides {x.stride()} on {x.device}")
    m = shape[0]
    if residual is not None:
        _same("residual", residual, (m, w.n_out), x.dtype, w.device)
    if y is not None:
        _same("y", y, (m, w.n_out), y.dtype, w.device)
    elif y_dtype is not None:
        y = x.new_empty((m, w.n_out), dtype=y_dtype)
    else:
        y = x.new_empty((m, w.n_out)) if residual is None else torch.empty_like(residual)
    status = lib.lk_w4_linear(w.packed_ptr, w.n_out, w.k_in, w.group, w.gated, x.data_ptr(), _code(x.dtype, _HALF), m,
                              x.stride(0) if m > 1 else w.k_in, None if residual is None else residual.data_ptr(),
                              y.data_ptr(), _code(y.dtype, _FLOAT), _raw_stream(w.index))
    if status:
        check(status)
    return y


def rmsnorm_gate_residual(y, x, w_post=None, gate=None, scale=1.0, w_pre=None, eps=1e-5, x_out=None, h=None,
                          stream=None):
    """x + scale * gate * (RMSNorm(y) * w_post), and RMSNorm of that * w_pre.

    y, x: [m, width]; w_post, w_pre: [width] (w_post None: y enters as it is;
    w_pre None: no second norm); gate: [width] or [m, width].  x_out may be x or
    y and h may be y.  Returns (x_out, h); h is None without w_pre.
    """
    dev = y.device
    if stream is not None or dev.index is None or dev.index != _current_device():
        return _enter(dev, stream, rmsnorm_gate_residual, y, x, w_post, gate, scale, w_pre, eps, x_out, h)
    dtype = y.dtype
    code = _code(dtype, _FLOAT)
    shape = y.shape
    if len(shape) != 2:
        raise ValueError("y: [m, width] is needed")
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
    status = lib.lk_rmsnorm_gate_residual(y.data_ptr(), x.data_ptr(), _ptr(w_post), _ptr(gate), per_row, _ptr(w_pre),
                                          code, m, width, scale, eps, x_out.data_ptr(), _ptr(h),
                                          _raw_stream(dev.index))
    if status:
        check(status)
    return x_out, h
