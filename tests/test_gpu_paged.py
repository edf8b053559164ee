"""Paged cache: append and decode attention against the float64 forms."""
import math

import pytest
import torch

from tests.paged_reference import HALF_STEP, Pages, attention, check

pytestmark = pytest.mark.gpu

BF, HF, I8 = torch.bfloat16, torch.float16, torch.int8


def run(pages, q, max_len=None, scale=None, accumulate=False, out_dtype=torch.float32, cache=None):
    import rank_latent_kv_lk_b200 as lk
    cache = cache or pages.cuda()
    max_len = max(pages.lens) if max_len is None else max_len
    out = lk.paged_decode_attn(cache, pages.table.cuda(), q.cuda(), pages.seq(), max_len, softmax_scale=scale,
                               accumulate=accumulate, out_dtype=out_dtype)
    return out, cache


def queries(pages, heads, dtype, scale=1.0):
    return (torch.randn(len(pages.lens), heads, pages.dim, generator=pages.g) * scale).to(dtype)


LENS = [0, 1, 15, 16, 17, 250]

CASES = [
    # lens, kv heads, group, dim, page, cache dtype, q dtype
    ([1], 1, 1, 16, 1, BF, BF),
    ([3], 1, 1, 32, 2, HF, HF),
    (LENS, 2, 1, 128, 16, BF, BF),
    (LENS, 2, 4, 128, 16, HF, HF),
    (LENS, 2, 8, 64, 4, HF, HF),
    (LENS, 1, 3, 80, 8, BF, BF),
    (LENS, 2, 5, 96, 32, HF, HF),
    (LENS, 1, 16, 128, 64, BF, BF),
    (LENS, 1, 12, 64, 16, BF, BF),
    (LENS, 1, 20, 112, 16, BF, BF),
    (LENS, 2, 6, 192, 16, BF, BF),
    (LENS, 1, 11, 256, 128, HF, HF),
    (LENS, 1, 128, 16, 1024, BF, BF),
    ([2049, 700, 1333], 3, 2, 128, 32, BF, BF),
    ([5000], 1, 1, 128, 16, BF, BF),
    ([0, 0], 2, 2, 64, 16, BF, BF),
    ([700, 0, 30, 655], 2, 2, 64, 16, BF, BF),          # longer than one CTA a unit takes, an empty one among them
    ([900, 1000], 2, 10, 96, 32, HF, HF),
    ([1500, 1, 0, 1499], 16, 2, 48, 8, HF, HF),
    ([600], 2, 9, 208, 16, BF, BF),
    ([520] * 40, 1, 1, 32, 128, HF, HF),
    ([530] * 5 + [0], 33, 1, 16, 16, I8, BF),
    (LENS, 2, 4, 128, 16, I8, BF),
    (LENS, 2, 4, 128, 16, I8, HF),
    (LENS, 1, 1, 16, 2, I8, BF),
    (LENS, 1, 9, 64, 32, I8, HF),
    (LENS, 2, 3, 80, 16, I8, BF),
    (LENS, 1, 16, 128, 64, I8, BF),
    (LENS, 1, 7, 192, 16, I8, HF),
    (LENS, 1, 8, 256, 16, I8, BF),
    ([3000, 1], 2, 4, 128, 64, I8, BF),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_decode_attention(case):
    lens, hk, group, dim, page, dt, qdt = case
    pages = Pages(lens, hk, dim, page, dt, seed=len(lens) * 100 + dim)
    q = queries(pages, hk * group, qdt)
    scale = 1 / math.sqrt(dim)
    want, tol, _, _ = attention(pages, q, scale)
    got, _ = run(pages, q)
    check(got, want, tol + 1e-30, "fp32 out")
    got, _ = run(pages, q, out_dtype=qdt)
    check(got, want, tol + HALF_STEP[qdt] * want.abs() + 2.0 ** -25, "16-bit out")


@pytest.mark.parametrize("case", [c for c in CASES if c[0] is not None][2::3],
                         ids=[str(i) for i in range(2, len(CASES), 3)])
def test_accumulated_weight(case):
    lens, hk, group, dim, page, dt, qdt = case
    pages = Pages(lens, hk, dim, page, dt, seed=7 + dim, mass=True, spread=2.0)
    q = queries(pages, hk * group, qdt)
    want, tol, mass, mtol = attention(pages, q, 1 / math.sqrt(dim), want_mass=True)
    got, cache = run(pages, q, accumulate=True)
    check(got, want, tol + 1e-30, "out")
    live = pages.live
    check(cache.mass.cpu()[live], mass[live], mtol[live] + 1e-30, "mass")
    assert torch.isnan(cache.mass.cpu()[~live]).all()  # rows of no token are left as they were


@pytest.mark.parametrize("dt,qdt", [(BF, BF), (HF, HF), (I8, BF)])
def test_sharp_scores_and_scale(dt, qdt):
    # one key dominates; a negative and a zero scale
    pages = Pages([333, 40], 2, 128, 16, dt, seed=3)
    q = queries(pages, 8, qdt, 6.0)
    for scale in (0.5, -0.25, 0.0):
        want, tol, _, _ = attention(pages, q, scale)
        got, _ = run(pages, q, scale=scale)
        check(got, want, tol + 1e-30, f"scale {scale}")


def test_masked_scores_of_minus_infinity():
    # keys that are -infinity in one dim: scores -infinity (q positive there), a head with nothing left gives zeros
    pages = Pages([40, 64], 1, 32, 16, BF, seed=5, mass=True)
    q = queries(pages, 2, BF)
    q[:, :, 0] = q[:, :, 0].abs() + 0.5
    flat = pages.table[0, 0].item()
    pages.k[flat, 0, :, 0] = -math.inf  # the first 16 tokens of sequence 0
    for p in pages.table[1, :4].tolist():
        pages.k[p, 0, :, 0] = -math.inf
    got, cache = run(pages, q, accumulate=True)
    k, v = pages.dense(0, 0)
    s = k @ q[0].to(torch.float64).t() / math.sqrt(32)
    p = torch.softmax(s, 0)
    assert torch.isinf(s[:16]).all()
    torch.testing.assert_close(got[0].cpu().double(), p.t() @ v, rtol=1e-4, atol=1e-5)
    assert (got[1] == 0).all()
    before, after = pages.rows(pages.mass, 1, 0), pages.rows(cache.mass.cpu(), 1, 0)
    assert torch.equal(before, after)
    assert torch.equal(pages.rows(pages.mass, 0, 0)[:16], pages.rows(cache.mass.cpu(), 0, 0)[:16])


def test_nan_stays_with_its_sequence_and_head():
    pages = Pages([100, 100], 2, 64, 16, HF, seed=9)
    pages.k[pages.table[0, 2], 1, 3, 5] = math.nan
    pages.v[pages.table[1, 1], 0, 0, 7] = math.inf
    q = queries(pages, 4, HF)
    got, _ = run(pages, q)
    got = got.cpu()
    assert torch.isnan(got[0, 2:]).all() and torch.isfinite(got[0, :2]).all()
    assert torch.isfinite(got[1, 2:]).all()
    assert not torch.isfinite(got[1, :2, 7]).any()
    rest = torch.arange(64) != 7
    assert torch.isfinite(got[1, :2][:, rest]).all()


def test_large_queries_in_an_int8_cache():
    # bf16 queries beyond fp16's range, and tiny ones
    for mag in (1e30, 1e-30):
        pages = Pages([77, 20], 1, 64, 16, I8, seed=2)
        q = queries(pages, 4, BF, mag)
        scale = 1 / mag / 8
        want, tol, _, _ = attention(pages, q, scale)
        got, _ = run(pages, q, scale=scale)
        check(got, want, tol + 1e-30, f"queries of {mag}")


def test_lengths_above_the_bound_are_cut():
    pages = Pages([100, 30], 1, 64, 16, BF, seed=4)
    q = queries(pages, 2, BF)
    got, _ = run(pages, q, max_len=48)
    pages.lens = [48, 30]
    want, tol, _, _ = attention(pages, q, 1 / 8)
    check(got, want, tol + 1e-30, "cut")


def test_strided_queries_and_shared_pages():
    import rank_latent_kv_lk_b200 as lk
    pages = Pages([64, 40], 2, 64, 16, BF, seed=6)
    pages.table[1, :3] = pages.table[0, :3]  # a shared prefix, read by both
    qkv = torch.randn(2, (4 + 2 + 2) * 64, generator=pages.g).to(BF)
    q = qkv[:, 64:64 + 256].view(2, 4, 64)
    want, tol, _, _ = attention(pages, q, 1 / 8)
    qd = qkv.cuda()[:, 64:64 + 256].view(2, 4, 64)
    got = lk.paged_decode_attn(pages.cuda(), pages.table.cuda(), qd, pages.seq(), 64, out_dtype=torch.float32)
    check(got, want, tol + 1e-30, "views")


def test_bad_pages_are_skipped_and_reported():
    import rank_latent_kv_lk_b200 as lk
    pages = Pages([40, 33], 1, 64, 16, BF, seed=8, mass=True)
    q = queries(pages, 2, BF)
    keep = [t for t in range(40) if not 16 <= t < 32]
    k, v = pages.dense(0, 0)
    p = torch.softmax(q[0].double() @ k[keep].t() / 8, -1)
    for bad in (-1, pages.n_pages, 2 ** 31 - 1):
        pages.table[0, 1] = bad
        got, _ = run(pages, q, accumulate=True)
        with pytest.raises(lk.LkError):
            lk.device_status()
        lk.device_status()  # reported once
        torch.testing.assert_close(got[0].cpu().double(), p @ v[keep], rtol=1e-3, atol=1e-4)


def test_results_do_not_depend_on_timing_or_stream():
    pages = Pages([3000, 17, 0, 2500], 2, 128, 16, BF, seed=11, mass=True)
    q = queries(pages, 8, BF)
    a, ca = run(pages, q, accumulate=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b, cb = run(pages, q, accumulate=True)
    side.synchronize()
    assert torch.equal(a, b)
    assert torch.equal(ca.mass.nan_to_num(-1), cb.mass.nan_to_num(-1))


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("dt,xdt", [(BF, BF), (HF, HF), (I8, BF), (I8, HF)])
@pytest.mark.parametrize("n_new,dim,page", [(1, 128, 16), (5, 80, 4), (33, 256, 1), (2, 16, 64)])
def test_append(dt, xdt, n_new, dim, page):
    import oracle as O
    import rank_latent_kv_lk_b200 as lk
    lens, hk = [0, 7, 31], 3
    pages = Pages(lens, hk, dim, page, dt, seed=n_new, mass=True, extra=n_new)
    cache = pages.cuda()
    qkv = torch.randn(3, n_new, (4 + 2 * hk) * dim, generator=pages.g).to(xdt)
    kn = qkv[..., 4 * dim:(4 + hk) * dim].unflatten(-1, (hk, dim))
    vn = qkv[..., (4 + hk) * dim:].unflatten(-1, (hk, dim))
    d = qkv.cuda()
    kd = d[..., 4 * dim:(4 + hk) * dim].unflatten(-1, (hk, dim))
    vd = d[..., (4 + hk) * dim:].unflatten(-1, (hk, dim))
    counts = [n_new, 0, n_new - 1]
    seq, nxt = pages.seq(), pages.seq() + 100
    new_len = torch.tensor([counts[0], -3, counts[2]], dtype=torch.int32, device="cuda")
    lk.paged_append(cache, pages.table.cuda(), kd, vd, seq, nxt, new_len=new_len)
    lk.device_status()
    assert seq.tolist() == [a + c for a, c in zip(lens, counts)]
    assert nxt.tolist() == [a + c + 100 for a, c in zip(lens, counts)]
    want = {n: getattr(pages, n).clone() for n in ("k", "v", "mass", "pos")}
    sc = {n: getattr(pages, n + "_scale") for n in ("k", "v")}
    for b in range(3):
        for i in range(counts[b]):
            t = lens[b] + i
            pg, off = pages.table[b, t // page].item(), t % page
            for n, x in (("k", kn), ("v", vn)):
                if dt is I8:
                    c, s = O.quantize_rows_i8(x[b, i].float().numpy())
                    want[n][pg, :, off] = torch.from_numpy(c)
                    sc[n][pg, :, off] = torch.from_numpy(s)
                else:
                    want[n][pg, :, off] = x[b, i]
            want["mass"][pg, :, off] = 0
            want["pos"][pg, :, off] = t + 100
    for n, x in want.items():
        torch.testing.assert_close(getattr(cache, n).cpu(), x, rtol=0, atol=0, equal_nan=True)
    if dt is I8:
        for n in ("k", "v"):
            torch.testing.assert_close(getattr(cache, n + "_scale").cpu(), sc[n], rtol=0, atol=0, equal_nan=True)


def test_append_that_does_not_fit_is_left_out():
    import rank_latent_kv_lk_b200 as lk
    pages = Pages([30, 5, 9], 2, 64, 16, BF, seed=1)  # two pages a sequence in the table
    cache = pages.cuda()
    kn = torch.randn(3, 3, 2, 64, device="cuda", dtype=BF)
    seq = torch.tensor([30, -2, 9], dtype=torch.int32, device="cuda")
    out = torch.full_like(seq, 99)
    lk.paged_append(cache, pages.table.cuda(), kn, kn, seq, seq_len_out=out)
    with pytest.raises(lk.LkError):
        lk.device_status()
    assert out.tolist() == [30, -2, 12]
    pages.lens = [30, 5, 9]
    for b, n in ((0, 30), (1, 5), (2, 9)):
        for h in range(2):
            assert torch.equal(pages.rows(cache.k.cpu(), b, h, n), pages.rows(pages.k, b, h, n))
    row = cache.k[pages.table[2, 0].item(), :, 9:12]
    assert torch.equal(row, kn[2].transpose(0, 1))


def test_append_then_attend_is_the_longer_cache():
    import rank_latent_kv_lk_b200 as lk
    pages = Pages([15, 16, 0, 100], 2, 128, 16, HF, seed=13, extra=1, mass=True)
    cache, table, seq = pages.cuda(), pages.table.cuda(), pages.seq()
    nxt = seq.clone()
    kn = torch.randn(4, 1, 2, 128, generator=pages.g).to(HF)
    vn = torch.randn(4, 1, 2, 128, generator=pages.g).to(HF)
    q = queries(pages, 8, HF)
    lk.paged_append(cache, table, kn.cuda(), vn.cuda(), seq, nxt)
    got = lk.paged_decode_attn(cache, table, q.cuda(), seq, 101, accumulate=True, out_dtype=torch.float32)
    for b in range(4):
        t = pages.lens[b]
        pg = pages.table[b, t // 16].item()
        pages.k[pg, :, t % 16], pages.v[pg, :, t % 16] = kn[b, 0], vn[b, 0]
        pages.mass[pg, :, t % 16] = 0
        pages.live[pg, :, t % 16] = True
        pages.lens[b] += 1
    want, tol, mass, mtol = attention(pages, q, 128 ** -0.5, want_mass=True)
    check(got, want, tol + 1e-30, "out")
    check(cache.mass.cpu()[pages.live], mass[pages.live], mtol[pages.live] + 1e-30, "mass")


@pytest.mark.parametrize("lens", [[2] * 64, [600, 513]], ids=["one CTA a unit", "split"])
def test_fp32_outputs_of_a_bf16_cache_keep_fp32_weights(lens):
    # Scores that are exact products: token 0 scores 0 and holds zeros, token 1 scores -q, the rest nothing.  Then
    # out = w v / (1 + w), w = exp(-q), q <= 1/4, and what is off relative to it, in units of 2^-22: the scaled score
    # (log2 e and one product, 0.36 2^-23 in log2) 0.13, the exponential 1, the weight's three terms 0.25 and their
    # sum 1.5, the sum of weights over warps and pieces 2, the quotient 0.5: below 6.  (Weights in two bf16 terms are
    # off by up to 2^-17.6, 21 of these.)
    pages = Pages(lens, 2, 16, 16, BF, seed=21)
    q = torch.zeros(len(lens), 8, 16)
    q[:, :, 0] = 0.05 + 0.2 * torch.rand(len(lens), 8, generator=pages.g)
    q = q.to(BF)
    pages.k[pages.live] = 0
    for b, n in enumerate(lens):
        for t in range(1, n):
            pages.k[pages.table[b, t // 16], :, t % 16, 0] = -1.0 if t == 1 else -1e38
        pages.v[pages.table[b, 0], :, 0] = 0
    got, _ = run(pages, q, scale=1.0)
    want = torch.zeros(len(lens), 8, 16, dtype=torch.float64)
    for b in range(len(lens)):
        for h in range(8):
            w = math.exp(-float(q[b, h, 0]))
            want[b, h] = w / (1 + w) * pages.dense(b, h // 4)[1][1]
    check(got, want, 6 * 2.0 ** -22 * want.abs() + 1e-30, "fp32 out")


MORE_WEIGHTS = [c for i, c in enumerate(CASES) if i % 3 != 2] + [
    # int8 and fp16 through the split and the join: one chunk of heads, two, an odd end, an empty sequence
    ([2000, 700], 1, 20, 128, 32, I8, BF),
    ([1100, 0, 531], 2, 11, 192, 16, I8, HF),
    ([3000, 1], 1, 40, 64, 64, I8, BF),
    ([2500, 513], 1, 17, 80, 4, HF, HF),
    ([5000], 1, 9, 256, 128, BF, BF),
]


@pytest.mark.parametrize("case", MORE_WEIGHTS, ids=[str(i) for i in range(len(MORE_WEIGHTS))])
def test_accumulated_weight_of_the_other_cases(case):
    test_accumulated_weight(case)


@pytest.mark.parametrize("dt", [BF, I8])
def test_rows_beyond_32_bits_of_bytes(dt):
    # the last pages of pools of 8.6 GB each, through append, attention and eviction: the same as on a small pool
    import rank_latent_kv_lk_b200 as lk
    dim, page, hk = 256, 64, 2
    big = 2 ** 33 // (dim * dt.itemsize * page * hk) + 7
    got = []
    for n_pages in (24, big):
        g = torch.Generator().manual_seed(5)
        shape = (n_pages, hk, page, dim)
        k, v = (torch.empty(shape, dtype=dt, device="cuda") for _ in range(2))
        rows = [torch.zeros(shape[:3], dtype=t, device="cuda") for t in (torch.float32, torch.int32)]
        sc = [torch.zeros(shape[:3], device="cuda") for _ in range(2)] if dt is I8 else [None, None]
        cache = lk.PagedKVCache.from_tensors(k, v, *sc, *rows)
        table = (n_pages - 24 + torch.randperm(24, generator=g)).to(torch.int32).view(2, 12).cuda()
        seq, nxt = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
        kn, vn = torch.randn(2, 2, 700, hk, dim, generator=g).to(BF).cuda()
        q = torch.randn(2, 8, dim, generator=g).to(BF).cuda()
        lk.paged_append(cache, table, kn, vn, seq, nxt)
        out = [lk.paged_decode_attn(cache, table, q, seq, 768, accumulate=True)]
        lk.paged_evict(cache, table, seq, nxt, 768, 320, window=32)
        out.append(lk.paged_decode_attn(cache, table, q, seq, 320))
        lk.device_status()
        assert seq.tolist() == [320, 320]
        ids = table[:, :5].long()
        got.append(out + [t[ids].clone() for t in (cache.k, cache.v, cache.mass, cache.pos)])
        del cache, k, v
    for a, b in zip(*got):
        assert torch.equal(a, b)
    torch.cuda.empty_cache()
