"""Eviction by accumulated attention weight against a sort."""
import math

import numpy as np
import pytest
import torch

from tests.paged_reference import Pages, evict

pytestmark = pytest.mark.gpu

BF, HF, I8 = torch.bfloat16, torch.float16, torch.int8


def expect(pages, next_pos, budget, window, n_sink):
    """The caches' rows after the call, and the written mass and pos."""
    names = ["k", "v"] + (["k_scale", "v_scale"] if pages.k_scale is not None else [])
    want = {n: getattr(pages, n).clone() for n in names + ["mass", "pos"]}
    page = pages.page
    for b, n in enumerate(pages.lens):
        for h in range(pages.kv_heads):
            src = evict(pages.rows(pages.mass, b, h).numpy(), pages.rows(pages.pos, b, h).numpy(), n, next_pos[b],
                        budget, window, n_sink)
            for t, s in enumerate(src):
                d = (pages.table[b, t // page].item(), h, t % page)
                f = (pages.table[b, s // page].item(), h, s % page)
                for x in want:
                    want[x][d] = getattr(pages, x)[f]
    return want


def compare(pages, cache, want, lens_before, budget):
    for n, x in want.items():
        torch.testing.assert_close(getattr(cache, n).cpu(), x, rtol=0, atol=0, equal_nan=True, msg=n)


CASES = [
    # lens, kv heads, dim, page, dtype, budget, window, sinks
    ([1], 1, 16, 1, BF, 1, 0, 0),
    ([2, 0, 1], 2, 32, 2, HF, 1, 1, 0),
    ([100, 64, 65, 3], 2, 64, 16, BF, 64, 8, 4),
    ([300, 299, 17], 3, 80, 32, HF, 150, 20, 2),
    ([500], 1, 128, 16, BF, 499, 0, 0),
    ([500], 1, 128, 16, BF, 1, 0, 0),
    ([257, 600], 2, 256, 64, I8, 200, 16, 4),
    ([300], 2, 64, 16, BF, 32, 100, 0),       # more protected than the budget
    ([5000, 4097], 1, 32, 128, BF, 1000, 64, 4),
    ([9000], 1, 16, 16, HF, 4500, 0, 1),
    ([700], 2, 16, 2, BF, 100, 300, 5),       # the same, pages of two rows
    ([20000, 70], 1, 16, 64, BF, 5000, 6000, 10),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
@pytest.mark.parametrize("kind", ["random", "ties", "special"])
def test_evict_in_place(case, kind):
    import rank_latent_kv_lk_b200 as lk
    lens, hk, dim, page, dt, budget, window, sinks = case
    pages = Pages(lens, hk, dim, page, dt, seed=budget, mass=True)
    if kind == "ties":
        pages.mass = torch.where(pages.live, (pages.mass * 3).floor(), pages.mass)
    if kind == "special":
        r = torch.rand(pages.mass.shape, generator=pages.g)
        m = pages.mass
        for lo, val in ((0.1, math.inf), (0.2, -math.inf), (0.3, math.nan), (0.4, -0.0), (0.5, 0.0), (0.55, -1.5)):
            m = torch.where(pages.live & (r < lo) & (r >= lo - 0.1), torch.tensor(val), m)
        pages.mass = m
    # positions in no order, as after an earlier eviction
    for b, n in enumerate(lens):
        for h in range(hk):
            perm = torch.randperm(n, generator=pages.g).to(torch.int32)
            for t in range(n):
                pages.pos[pages.table[b, t // page], h, t % page] = perm[t]
    cache, seq = pages.cuda(), pages.seq()
    nxt = [n + (b % 2) * 5 for b, n in enumerate(lens)]
    want = expect(pages, nxt, budget, window, sinks)
    lk.paged_evict(cache, pages.table.cuda(), seq, torch.tensor(nxt, dtype=torch.int32, device="cuda"), max(lens),
                   budget, window=window, n_sink=sinks)
    lk.device_status()
    assert seq.tolist() == [min(n, budget) for n in lens]
    compare(pages, cache, want, lens, budget)


@pytest.mark.parametrize("budget", [199, 200, 201, 399, 400, 401])
def test_weights_of_a_few_magnitudes(budget):
    # the limit lies at or beside the end of a bin of equal leading bits: 200 weights each around 1, 2^-40 and 2^-80
    import rank_latent_kv_lk_b200 as lk
    n, page = 600, 16
    g = torch.Generator().manual_seed(budget)
    mag = torch.tensor([1.0, 2.0 ** -40, 2.0 ** -80]).repeat_interleave(200)[torch.randperm(n, generator=g)]
    shape = (-(-n // page), 1, page)
    mass, pos = torch.zeros(shape), torch.zeros(shape, dtype=torch.int32)
    mass.view(-1)[:n] = mag * (1 + torch.randint(0, 50, (n,), generator=g) * 2.0 ** -20)
    pos.view(-1)[:n] = torch.arange(n, dtype=torch.int32)
    k = torch.randn(shape + (16,), generator=g).to(BF)
    cache = lk.PagedKVCache.from_tensors(k.cuda(), k.cuda(), None, None, mass.cuda(), pos.cuda())
    seq = torch.tensor([n], dtype=torch.int32, device="cuda")
    table = torch.arange(shape[0], dtype=torch.int32, device="cuda")[None]
    lk.paged_evict(cache, table, seq, seq.clone(), n, budget)
    src = torch.from_numpy(np.asarray(evict(mass.view(-1)[:n].numpy(), pos.view(-1)[:n].numpy(), n, n, budget, 0, 0)))
    assert seq.tolist() == [budget]
    for got, was in ((cache.mass, mass), (cache.pos, pos), (cache.k, k), (cache.v, k)):
        assert torch.equal(got.cpu().flatten(0, 2)[:budget], was.flatten(0, 2)[src])


@pytest.mark.parametrize("lens,budget", [([70000], 30000), ([60000, 100], 50000), ([30001], 7), ([2000, 100001], 1999),
                                         ([66000], 33000)])
def test_evict_long_sequences(lens, budget):
    # longer than shared memory holds keys for
    import rank_latent_kv_lk_b200 as lk
    B, page, dim = len(lens), 512, 16
    width = -(-max(lens) // page)
    g = torch.Generator().manual_seed(1)
    shape = (B * width, 1, page, dim)
    k = torch.randn(shape, generator=g).to(BF)
    v = torch.randn(shape, generator=g).to(BF)
    mass = (torch.rand(shape[:3], generator=g) * 5000).floor()
    pos = torch.arange(width * page, dtype=torch.int32).repeat(B).view(shape[:3])
    table = torch.randperm(B * width, generator=g).to(torch.int32).view(B, width)
    pos[table.flatten().long()] = pos.clone()
    if lens == [66000]:  # the upper half of the slots is wanted: whole rounds of words move
        wanted = torch.arange(width * page).view(width, page) >= 33000
        mass[table[0].long(), 0] = torch.where(wanted, 1.0 + mass[table[0].long(), 0], 0.0)
    cache = lk.PagedKVCache.from_tensors(k.cuda(), v.cuda(), None, None, mass.cuda(), pos.cuda())
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out_m, out_p = torch.zeros_like(cache.mass), torch.zeros_like(cache.pos)
    out_s = torch.zeros_like(seq)
    lk.paged_evict(cache, table.cuda(), seq, seq + 3, max(lens), budget, window=100, n_sink=4, mass_out=out_m,
                   pos_out=out_p, seq_len_out=out_s)
    lk.device_status()
    assert seq.tolist() == lens and out_s.tolist() == [min(n, budget) for n in lens]
    assert torch.equal(cache.mass.cpu(), mass) and torch.equal(cache.pos.cpu(), pos)
    for b, n in enumerate(lens):
        ids = table[b].long()
        flat = [x[ids, 0].flatten(0, 1) for x in (mass, pos, k, v)]
        src = evict(flat[0].numpy(), flat[1].numpy(), n, n + 3, budget, 100, 4)
        got = [x.cpu()[ids, 0].flatten(0, 1) for x in (out_m, out_p, cache.k, cache.v)]
        src = torch.from_numpy(np.asarray(src))
        for x, y in zip(got, flat):
            assert torch.equal(x[:len(src)], y[src])
        assert torch.equal(got[2][len(src):], flat[2][len(src):])  # rows moved away from stay
        assert (got[0][len(src):] == 0).all()


@pytest.mark.parametrize("dt", [BF, I8])
@pytest.mark.parametrize("lens,budget", [([260, 100, 300], 200), ([900, 10], 400)])
def test_outputs_apart_and_in_place_agree(dt, lens, budget):
    # the lengths in another array or in place; few rows that move (one launch) and many
    import rank_latent_kv_lk_b200 as lk
    got = []
    for apart in (False, True):
        pages = Pages(lens, 2, 48, 16, dt, seed=4, mass=True)
        cache, seq = pages.cuda(), pages.seq()
        kw = {}
        if apart:
            kw = dict(mass_out=torch.full_like(cache.mass, -1), pos_out=torch.full_like(cache.pos, -1),
                      seq_len_out=torch.full_like(seq, -1))
        lk.paged_evict(cache, pages.table.cuda(), seq, seq + 2, max(lens), budget, window=5, n_sink=3, **kw)
        if apart:
            assert seq.tolist() == lens
            assert torch.equal(cache.mass.cpu().nan_to_num(9), pages.mass.nan_to_num(9))
            seq, cache.mass, cache.pos = kw["seq_len_out"], kw["mass_out"], kw["pos_out"]
        assert seq.tolist() == [min(n, budget) for n in lens]
        got.append([[pages.rows(t.cpu(), b, h, min(n, budget)) for t in (cache.k, cache.v, cache.mass, cache.pos)]
                    for b, n in enumerate(lens) for h in range(2)])
    for a, b in zip(*got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_evict_skips_and_reports_bad_pages():
    import rank_latent_kv_lk_b200 as lk
    pages = Pages([64, 20], 1, 32, 16, BF, seed=2, mass=True)
    pages.table[0, 1] = pages.n_pages
    pages.table[0, 3] = -1
    cache, seq = pages.cuda(), pages.seq()
    lk.paged_evict(cache, pages.table.cuda(), seq, seq.clone(), 64, 24, window=2)
    with pytest.raises(lk.LkError):
        lk.device_status()
    assert seq.tolist() == [24, 20]
    for h in range(1):
        assert torch.equal(pages.rows(cache.k.cpu(), 1, h, 20), pages.rows(pages.k, 1, h, 20))


def test_lengths_between_the_calls_of_a_batch():
    # nothing leaves: lengths equal to and below the budget, none at all
    import rank_latent_kv_lk_b200 as lk
    pages = Pages([64, 0, 10], 2, 64, 16, HF, seed=3, mass=True)
    cache, seq = pages.cuda(), pages.seq()
    lk.paged_evict(cache, pages.table.cuda(), seq, seq.clone(), 64, 64)
    lk.paged_evict(cache, pages.table.cuda(), seq, seq.clone(), 64, 1000)
    lk.device_status()
    assert seq.tolist() == [64, 0, 10]
    for n in ("k", "v", "mass", "pos"):
        torch.testing.assert_close(getattr(cache, n).cpu(), getattr(pages, n), rtol=0, atol=0, equal_nan=True)


def test_outputs_apart_take_the_caches_place():
    # an eviction into arrays of their own, which then become the cache's: what follows is what follows one in place
    import rank_latent_kv_lk_b200 as lk
    caches = []
    for apart in (False, True):
        pages = Pages([260, 100, 300], 2, 64, 16, BF, seed=6, mass=True, extra=1)
        cache, seq, table = pages.cuda(), pages.seq(), pages.table.cuda()
        nxt = seq.clone()
        g = torch.Generator().manual_seed(1)
        q = torch.randn(3, 4, 64, generator=g).to(BF).cuda()
        k, v = torch.randn(2, 3, 1, 2, 64, generator=g).to(BF).cuda()
        if apart:
            m, p = cache.mass.clone(), cache.pos.clone()
            lk.paged_evict(cache, table, seq, nxt, 301, 90, window=5, mass_out=m, pos_out=p)
            cache.mass, cache.pos = m, p
            assert cache.mass is m and cache.pos is p
        else:
            lk.paged_evict(cache, table, seq, nxt, 301, 90, window=5)
        lk.paged_append(cache, table, k, v, seq, nxt)
        out = lk.paged_decode_attn(cache, table, q, seq, 301, accumulate=True)
        lk.paged_evict(cache, table, seq, nxt, 301, 50, window=5)
        caches.append((pages, cache, out, seq.tolist()))
    (pages, a, out_a, n_a), (_, b, out_b, n_b) = caches
    assert torch.equal(out_a, out_b) and n_a == n_b == [50] * 3
    for name in ("k", "v", "mass", "pos"):
        x, y = getattr(a, name).cpu(), getattr(b, name).cpu()
        for s in range(3):
            for h in range(2):
                assert torch.equal(pages.rows(x, s, h, 50), pages.rows(y, s, h, 50)), name


def test_tensors_of_a_cache_and_a_weight():
    import rank_latent_kv_lk_b200 as lk
    cache = lk.PagedKVCache(8, 16, 2, 64, mass=True)
    assert (cache.n_pages, cache.n_kv_heads, cache.page_size, cache.head_dim) == (8, 2, 16, 64)
    before = cache.k, cache.mass
    with pytest.raises(ValueError):
        cache.mass = None                                  # positions without weights
    with pytest.raises(ValueError):
        cache.k = torch.zeros(9, 2, 16, 64, dtype=BF, device="cuda")
    with pytest.raises(TypeError):
        cache.mass = cache.mass.half()
    with pytest.raises(ValueError):
        cache.v = cache.v.cpu()
    with pytest.raises(AttributeError):
        cache.page_size = 32
    assert cache.k is before[0] and cache.mass is before[1]
    # storage changed in place: the calls see it, and refuse sizes that no longer fit
    table = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    seq, nxt = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    one = torch.ones(1, 1, 2, 64, dtype=BF, device="cuda")
    cache.v.set_(torch.full_like(cache.v, 3))
    lk.paged_append(cache, table, one, one, seq, nxt)
    out = lk.paged_decode_attn(cache, table, one[:, 0], seq, 32)
    assert (out == 1).all() and (cache.v[0, :, 0] == 1).all() and (cache.v[0, :, 1] == 3).all()
    cache.pos.resize_(8, 2, 8)
    for call in (lambda: lk.paged_append(cache, table, one, one, seq, nxt),
                 lambda: lk.paged_decode_attn(cache, table, one[:, 0], seq, 32),
                 lambda: lk.paged_evict(cache, table, seq, nxt, 32, 8)):
        with pytest.raises(ValueError):
            call()
    w = lk.W4Weight(torch.zeros(16, 32, dtype=torch.uint8, device="cuda"),
                    torch.zeros(16, 1, dtype=torch.float16, device="cuda"))
    with pytest.raises(AttributeError):
        w.packed = torch.zeros(1)
    w.packed.resize_(16)
    with pytest.raises(ValueError):
        lk.w4_linear(w, torch.zeros(1, 64, dtype=BF, device="cuda"))


# 1025 to 4096 slots: the selecting kernel of 512 threads; lens, kv heads, dim, page, dtype, budget, window, sinks
MIDDLE = [
    ([1025, 900, 3], 2, 32, 16, BF, 900, 16, 4),       # 125 rows can move: one launch beside the lengths
    ([2112, 2049], 2, 64, 64, HF, 2048, 128, 4),
    ([4096, 4095, 0], 1, 16, 32, I8, 3900, 64, 0),
    ([1025], 1, 128, 2, BF, 300, 20, 4),               # many rows move
    ([4096, 1500], 2, 32, 128, HF, 1000, 64, 4),
    ([3000], 1, 48, 16, I8, 1400, 0, 0),
    ([2112, 700], 1, 16, 16, BF, 500, 900, 30),        # more protected than the budget
    ([4000, 4000], 1, 16, 1, BF, 3990, 4000, 2),
]


@pytest.mark.parametrize("case", MIDDLE, ids=[str(i) for i in range(len(MIDDLE))])
@pytest.mark.parametrize("kind", ["random", "ties", "special"])
def test_evict_sequences_of_middle_length(case, kind):
    test_evict_in_place(case, kind)


@pytest.mark.parametrize("case", MIDDLE, ids=[str(i) for i in range(len(MIDDLE))])
@pytest.mark.parametrize("kind", ["random", "ties"])
@pytest.mark.parametrize("lengths_apart", [False, True])
def test_evict_sequences_of_middle_length_into_outputs_apart(case, kind, lengths_apart):
    import rank_latent_kv_lk_b200 as lk
    lens, hk, dim, page, dt, budget, window, sinks = case
    pages = Pages(lens, hk, dim, page, dt, seed=budget + 1, mass=True)
    if kind == "ties":
        pages.mass = torch.where(pages.live, (pages.mass * 3).floor(), pages.mass)
    want = expect(pages, lens, budget, window, sinks)
    cache, seq = pages.cuda(), pages.seq()
    m, p = torch.full_like(cache.mass, -1), torch.full_like(cache.pos, -1)
    out = torch.full_like(seq, -1) if lengths_apart else seq
    lk.paged_evict(cache, pages.table.cuda(), seq, seq.clone(), max(lens), budget, window=window, n_sink=sinks,
                   mass_out=m, pos_out=p, seq_len_out=out)
    lk.device_status()
    assert out.tolist() == [min(n, budget) for n in lens]
    if lengths_apart:
        assert seq.tolist() == lens
    assert torch.equal(cache.mass.cpu().nan_to_num(9), pages.mass.nan_to_num(9))
    assert torch.equal(cache.pos.cpu(), pages.pos)
    for n in [x for x in want if x not in ("mass", "pos")]:
        torch.testing.assert_close(getattr(cache, n).cpu(), want[n], rtol=0, atol=0, equal_nan=True, msg=n)
    kept = torch.zeros_like(pages.live)
    for b, n in enumerate(lens):
        for t in range(min(n, budget)):
            kept[pages.table[b, t // page], :, t % page] = True
    for got, n in ((m.cpu(), "mass"), (p.cpu(), "pos")):
        assert torch.equal(got[kept], want[n][kept]), n
        assert (got[~kept] == -1).all(), n
