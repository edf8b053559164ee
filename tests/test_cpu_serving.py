"""CPU-only checks of the serving operators' C ABI (lk_serving.h): every symbol
is exported and every bad argument is refused on the host, before CUDA is
touched (a call that got through would report LK_ERR_CUDA here)."""
import ctypes as C
import os
import re
import shutil
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000  # 256-byte aligned fake device address


def at(i):
    return FAKE + i * 0x100000


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    from rank_latent_kv_lk_b200 import _lib
    return _lib


def test_every_declared_symbol_is_exported(L):
    with open(os.path.join(ROOT, "include", "lk_serving.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(lk_[a-z0-9_]+)\s*\(", text)))
    assert len(names) == 9
    for n in names:
        assert hasattr(L.lib, n), n


def desc(L, n_pages=8, page_size=16, heads=2, dim=64, dtype=None, k=at(0), v=at(1), ks=None, vs=None, mass=None,
         pos=None):
    return L.PagedCacheDesc(n_pages, page_size, heads, dim, L.LK_BF16 if dtype is None else dtype, k, v, ks, vs, mass,
                            pos)


BAD_CACHES = [
    (dict(dtype=0), "LK_ERR_DTYPE"), (dict(dtype=4), "LK_ERR_DTYPE"), (dict(n_pages=0), "LK_ERR_SHAPE"),
    (dict(page_size=0), "LK_ERR_SHAPE"), (dict(page_size=24), "LK_ERR_SHAPE"), (dict(page_size=2048), "LK_ERR_SHAPE"),
    (dict(heads=0), "LK_ERR_SHAPE"), (dict(heads=129), "LK_ERR_SHAPE"), (dict(dim=24), "LK_ERR_SHAPE"),
    (dict(dim=272), "LK_ERR_SHAPE"), (dict(dim=0), "LK_ERR_SHAPE"),
    (dict(n_pages=1 << 27, page_size=16), "LK_ERR_SHAPE"),                 # 2^31 rows and more
    (dict(k=None), "LK_ERR_INVALID_ARG"), (dict(v=None), "LK_ERR_INVALID_ARG"), (dict(k=at(0) + 8), "LK_ERR_ALIGN"),
    (dict(ks=at(2), vs=at(3)), "LK_ERR_INVALID_ARG"),                      # scales of a 16-bit cache
    (dict(dtype=3), "LK_ERR_INVALID_ARG"), (dict(dtype=3, ks=at(2)), "LK_ERR_INVALID_ARG"),
    (dict(mass=at(2)), "LK_ERR_INVALID_ARG"), (dict(pos=at(2)), "LK_ERR_INVALID_ARG"),
    (dict(mass=at(2) + 4, pos=at(3)), "LK_ERR_ALIGN"),
]


def decode(L, d=None, table=at(4), batch=2, width=4, q=at(5), qdt=None, heads=4, q_stride=None, seq=at(6), max_len=40,
           scale=0.1, acc=0, out=at(7), odt=None, ws=at(8), ws_bytes=1 << 26):
    d = desc(L) if d is None else d
    return L.lib.lk_paged_decode_attn(C.byref(d), table, batch, width, q, L.LK_BF16 if qdt is None else qdt, heads,
                                      heads * d.head_dim if q_stride is None else q_stride, seq, max_len, scale, acc,
                                      out, L.LK_F32 if odt is None else odt, ws, ws_bytes, None)


def append(L, d=None, table=at(4), batch=2, width=4, k=at(5), v=at(6), dt=None, stride=None, n_new=1, new_len=None,
           seq=at(7), seq_out=at(7), nxt=None, nxt_out=None):
    d = desc(L) if d is None else d
    return L.lib.lk_paged_append(C.byref(d), table, batch, width, k, v, L.LK_BF16 if dt is None else dt,
                                 d.n_kv_heads * d.head_dim if stride is None else stride, n_new, new_len, seq, seq_out,
                                 nxt, nxt_out, None)


def evict(L, d=None, table=at(4), batch=2, width=4, seq=at(5), nxt=at(6), max_len=40, budget=16, window=0, sink=0,
          mass=at(2), pos=at(3), seq_out=at(5), ws=at(8), ws_bytes=1 << 26):
    d = desc(L, mass=at(2), pos=at(3)) if d is None else d
    return L.lib.lk_paged_evict(C.byref(d), table, batch, width, seq, nxt, max_len, budget, window, sink, mass, pos,
                                seq_out, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [decode, append, evict])
@pytest.mark.parametrize("bad,status", BAD_CACHES, ids=[str(b[0]) for b in BAD_CACHES])
def test_bad_caches(L, call, bad, status):
    bad = dict(bad)
    if call is evict and not {"mass", "pos"} & set(bad):
        bad.update(mass=at(2), pos=at(3))
    assert call(L, desc(L, **bad)) == getattr(L, status)
    assert L.lib.lk_last_error()


def test_decode_refusals(L):
    E = L
    i8 = desc(L, dtype=L.LK_I8, ks=at(2), vs=at(3))
    assert decode(L, table=None) == E.LK_ERR_INVALID_ARG
    for name in ("q", "seq", "out"):
        assert decode(L, **{name: None}) == E.LK_ERR_INVALID_ARG, name
    assert decode(L, batch=0) == E.LK_ERR_SHAPE
    assert decode(L, width=0) == E.LK_ERR_SHAPE
    assert decode(L, max_len=65) == E.LK_ERR_SHAPE            # beyond the table
    assert decode(L, width=(1 << 26) + 1) == E.LK_ERR_SHAPE   # slots beyond 2^30
    assert decode(L, max_len=-1) == E.LK_ERR_SHAPE
    assert decode(L, heads=3) == E.LK_ERR_SHAPE
    assert decode(L, heads=0) == E.LK_ERR_SHAPE
    assert decode(L, heads=130) == E.LK_ERR_SHAPE
    assert decode(L, qdt=L.LK_F16) == E.LK_ERR_DTYPE          # not the cache's
    assert decode(L, qdt=L.LK_F32) == E.LK_ERR_DTYPE
    assert decode(L, i8, qdt=L.LK_I8) == E.LK_ERR_DTYPE
    assert decode(L, odt=L.LK_I8) == E.LK_ERR_DTYPE
    assert decode(L, q_stride=252) == E.LK_ERR_ALIGN
    assert decode(L, q_stride=248) == E.LK_ERR_SHAPE
    assert decode(L, q=at(5) + 2) == E.LK_ERR_ALIGN
    assert decode(L, out=at(7) + 8) == E.LK_ERR_ALIGN
    assert decode(L, out=at(5)) == E.LK_ERR_INVALID_ARG       # over q
    assert decode(L, out=at(5) + 1008) == E.LK_ERR_INVALID_ARG
    assert decode(L, acc=1) == E.LK_ERR_INVALID_ARG           # a cache without mass
    assert decode(L, acc=2) == E.LK_ERR_INVALID_ARG
    assert decode(L, scale=float("nan")) == E.LK_ERR_INVALID_ARG
    assert decode(L, ws=None) == E.LK_ERR_WORKSPACE
    assert decode(L, ws_bytes=100) == E.LK_ERR_WORKSPACE
    assert decode(L, ws=at(8) + 128) == E.LK_ERR_ALIGN
    need = L.lib.lk_paged_decode_workspace_bytes(C.byref(desc(L)), 2, 4, 40, 0)
    assert need > 0 and decode(L, ws_bytes=need - 1) == E.LK_ERR_WORKSPACE
    m = desc(L, mass=at(2), pos=at(3))
    for n in (0, 40, 4000):                                   # one launch, two launches
        less = L.lib.lk_paged_decode_workspace_bytes(C.byref(m), 2, 4, n, 0)
        more = L.lib.lk_paged_decode_workspace_bytes(C.byref(m), 2, 4, n, 1)
        scores = 2 * 2 * -(-n // 16) * 2 * 16 * 4             # blocks of 16 tokens, 2 heads a group
        assert less > 0 and more in (max(scores, 256), less + scores)


def test_append_refusals(L):
    E = L
    m = desc(L, mass=at(2), pos=at(3))
    assert append(L, table=None) == E.LK_ERR_INVALID_ARG
    for name in ("k", "v", "seq", "seq_out"):
        assert append(L, **{name: None}) == E.LK_ERR_INVALID_ARG, name
    assert append(L, dt=L.LK_F16) == E.LK_ERR_DTYPE
    assert append(L, dt=L.LK_F32) == E.LK_ERR_DTYPE
    assert append(L, n_new=0) == E.LK_ERR_SHAPE
    assert append(L, batch=0) == E.LK_ERR_SHAPE
    assert append(L, stride=120) == E.LK_ERR_SHAPE
    assert append(L, stride=132) == E.LK_ERR_ALIGN
    assert append(L, k=at(5) + 4) == E.LK_ERR_ALIGN
    assert append(L, m) == E.LK_ERR_INVALID_ARG               # mass without positions
    assert append(L, m, nxt=at(9)) == E.LK_ERR_INVALID_ARG
    assert append(L, nxt=at(9), nxt_out=at(9)) == E.LK_ERR_INVALID_ARG
    assert append(L, seq_out=at(7) + 4) == E.LK_ERR_INVALID_ARG           # lengths shifted by one
    assert append(L, m, nxt=at(7), nxt_out=at(7)) == E.LK_ERR_INVALID_ARG  # lengths and positions in one array
    assert append(L, new_len=at(7)) == E.LK_ERR_INVALID_ARG


def test_evict_refusals(L):
    E = L
    assert evict(L, desc(L)) == E.LK_ERR_INVALID_ARG          # no mass
    for name in ("table", "seq", "nxt", "mass", "pos", "seq_out"):
        assert evict(L, **{name: None}) == E.LK_ERR_INVALID_ARG, name
    assert evict(L, budget=0) == E.LK_ERR_SHAPE
    assert evict(L, window=-1) == E.LK_ERR_SHAPE
    assert evict(L, sink=-1) == E.LK_ERR_SHAPE
    assert evict(L, max_len=65) == E.LK_ERR_SHAPE
    assert evict(L, mass=at(9)) == E.LK_ERR_INVALID_ARG       # one in place, one not
    assert evict(L, mass=at(9) + 4, pos=at(10)) == E.LK_ERR_ALIGN
    assert evict(L, mass=at(2) + 64, pos=at(10)) == E.LK_ERR_INVALID_ARG  # partly over the cache's
    assert evict(L, mass=at(9), pos=at(9) + 512) == E.LK_ERR_INVALID_ARG  # over each other
    assert evict(L, mass=at(3), pos=at(9)) == E.LK_ERR_INVALID_ARG
    assert evict(L, seq_out=at(5) + 4) == E.LK_ERR_INVALID_ARG
    assert evict(L, seq_out=at(6)) == E.LK_ERR_INVALID_ARG    # over the positions
    assert evict(L, ws_bytes=8) == E.LK_ERR_WORKSPACE
    assert evict(L, ws=at(8) + 16) == E.LK_ERR_ALIGN


def w4(L, packed=at(0), n=32, k=128, group=64, gated=0, x=at(1), xdt=None, m=2, stride=128, res=None, y=at(2), ydt=None):
    return L.lib.lk_w4_linear(packed, n, k, group, gated, x, L.LK_BF16 if xdt is None else xdt, m, stride, res, y,
                              L.LK_BF16 if ydt is None else ydt, None)


def test_w4_refusals(L):
    E = L
    assert w4(L, group=16) == E.LK_ERR_SHAPE
    assert w4(L, k=96) == E.LK_ERR_SHAPE
    assert w4(L, n=0) == E.LK_ERR_SHAPE
    assert w4(L, m=-1) == E.LK_ERR_SHAPE
    assert w4(L, xdt=L.LK_F32) == E.LK_ERR_DTYPE
    assert w4(L, ydt=L.LK_I8) == E.LK_ERR_DTYPE
    for name in ("packed", "x", "y"):
        assert w4(L, **{name: None}) == E.LK_ERR_INVALID_ARG, name
    assert w4(L, stride=120) == E.LK_ERR_SHAPE
    assert w4(L, stride=132) == E.LK_ERR_ALIGN
    assert w4(L, gated=1, res=at(3)) == E.LK_ERR_UNSUPPORTED
    assert w4(L, gated=2) == E.LK_ERR_INVALID_ARG
    assert w4(L, res=at(2), ydt=L.LK_F32) == E.LK_ERR_INVALID_ARG
    assert w4(L, res=at(2) + 16) == E.LK_ERR_INVALID_ARG      # partly over y
    assert w4(L, y=at(1) + 256) == E.LK_ERR_INVALID_ARG       # over x
    assert w4(L, packed=at(0) + 16) == E.LK_ERR_ALIGN
    assert w4(L, x=at(1) + 2) == E.LK_ERR_ALIGN

    def pack(codes=at(0), scales=at(1), uc=None, us=None, n=32, k=128, group=64, out=at(2), size=1 << 20):
        return L.lib.lk_w4_pack(codes, scales, uc, us, n, k, group, out, size, None)

    need = L.lib.lk_w4_packed_bytes(32, 128, 64, 0)
    assert need == 32 * 128 // 2 + 32 * 2 * 2 and L.lib.lk_w4_packed_bytes(32, 128, 64, 1) == 2 * need
    assert L.lib.lk_w4_packed_bytes(32, 128, 48, 0) == 0
    assert pack(codes=None) == E.LK_ERR_INVALID_ARG
    assert pack(uc=at(3)) == E.LK_ERR_INVALID_ARG
    assert pack(codes=at(0) + 1) == E.LK_ERR_ALIGN
    assert pack(out=at(2) + 16) == E.LK_ERR_ALIGN
    assert pack(size=need - 1) == E.LK_ERR_WORKSPACE
    assert pack(group=256, k=256) == E.LK_ERR_SHAPE


def test_norm_refusals(L):
    E = L

    def norm(y=at(0), x=at(1), wp=None, gate=None, per_row=0, wq=None, dt=None, m=2, width=64, scale=1.0, eps=1e-5,
             xo=at(2), h=None):
        return L.lib.lk_rmsnorm_gate_residual(y, x, wp, gate, per_row, wq, L.LK_BF16 if dt is None else dt, m, width,
                                              scale, eps, xo, h, None)

    assert norm(dt=L.LK_I8) == E.LK_ERR_DTYPE
    assert norm(width=0) == E.LK_ERR_SHAPE
    assert norm(width=32769) == E.LK_ERR_SHAPE
    assert norm(m=-1) == E.LK_ERR_SHAPE
    for name in ("y", "x", "xo"):
        assert norm(**{name: None}) == E.LK_ERR_INVALID_ARG, name
    assert norm(wq=at(3)) == E.LK_ERR_INVALID_ARG
    assert norm(h=at(3)) == E.LK_ERR_INVALID_ARG
    assert norm(wq=at(3), h=at(1)) == E.LK_ERR_INVALID_ARG    # h over x
    assert norm(wq=at(3), h=at(2)) == E.LK_ERR_INVALID_ARG    # h over x_out
    assert norm(xo=at(0) + 2) == E.LK_ERR_INVALID_ARG         # partly over y
    assert norm(wp=at(2) + 64) == E.LK_ERR_INVALID_ARG        # a weight under an output
    assert norm(gate=at(2), per_row=1) == E.LK_ERR_INVALID_ARG
    assert norm(wq=at(3), h=at(2) + 128) == E.LK_ERR_INVALID_ARG
    assert norm(per_row=2) == E.LK_ERR_INVALID_ARG
    assert norm(eps=-1.0) == E.LK_ERR_INVALID_ARG
    assert norm(eps=float("nan")) == E.LK_ERR_INVALID_ARG
    assert norm(scale=float("nan")) == E.LK_ERR_INVALID_ARG
    assert norm(y=at(0) + 1) == E.LK_ERR_ALIGN


def test_wrappers_refuse_tensors_of_the_host(L):
    import rank_latent_kv_lk_b200 as lk
    k = torch.zeros(2, 1, 16, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lk.PagedKVCache.from_tensors(k, k)
    with pytest.raises(ValueError):
        lk.rmsnorm_gate_residual(k[0, 0], k[0, 0])
    with pytest.raises(ValueError):
        lk.W4Weight(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.float16))


def test_the_latent_layer_does_without_the_serving_binding(L):
    # as where the binding does not fit the installed torch: W8A8DecoderLayer needs only liblk.so
    code = ("import sys; sys.modules['rank_latent_kv_lk_b200._serving_ext'] = None\n"
            "from rank_latent_kv_lk_b200.layer import W8A8DecoderLayer, W4PagedDecoderLayer\n"
            "try:\n    W4PagedDecoderLayer({}, 8, 2, 64, 8, 16)\n"
            "except ImportError:\n    print('refused')\n")
    p = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
    assert p.stdout.split() == ["refused"]


def test_the_binding_is_built_again_for_another_torch(L, tmp_path, monkeypatch):
    import importlib.metadata
    import importlib.util

    import __graft_entry__
    b = __graft_entry__._load_builder()
    shutil.copy2(b.EXT, tmp_path / "ext.so")
    monkeypatch.setattr(b, "EXT", str(tmp_path / "ext.so"))
    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    built = []

    def compiler(cmd, **kw):
        built.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b.subprocess, "run", compiler)
    b._build_ext(True, False)
    b._build_ext(False, False)
    assert len(built) == 1                                    # nothing changed
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.1")
    b._build_ext(False, False)
    b._build_ext(False, False)
    assert len(built) == 2
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda n, *a: None if n == "torch" else find(n, *a))
    b._build_ext(True, False)                                 # no torch: the library alone
    assert len(built) == 2


def test_workspaces_of_sequences_longer_than_any_table(L):
    # a table has at most 2^30 slots: no size for more, and none that wrapped around
    m = desc(L, mass=at(2), pos=at(3))
    for n, known in ((1 << 30, True), ((1 << 30) + 1, False), (2 ** 31 - 1, False)):
        sizes = [L.lib.lk_paged_decode_workspace_bytes(C.byref(m), 2, 4, n, acc) for acc in (0, 1)]
        sizes.append(L.lib.lk_paged_evict_workspace_bytes(C.byref(m), 2, n, 64))
        assert all((s > 0) == known for s in sizes), (n, sizes)
    # scores of 2^30 slots; keys and bits of as many for eviction
    assert L.lib.lk_paged_decode_workspace_bytes(C.byref(m), 2, 4, 1 << 30, 1) >= 2 * 4 * 2 ** 30 * 4
    assert L.lib.lk_paged_evict_workspace_bytes(C.byref(m), 2, 1 << 30, 64) >= 4 * 2 ** 30 * 4
