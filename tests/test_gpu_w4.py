"""4-bit products against float64."""
import pytest
import torch

from tests.paged_reference import F64, HALF_STEP, check

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def weights(n, k, group, g):
    codes = torch.randint(0, 256, (n, k // 2), generator=g).to(torch.uint8)  # every nibble, -8 among them
    scales = (torch.randn(n, k // group, generator=g) / k ** 0.5).to(HF)     # of both signs
    scales[0, 0] = 0
    return codes, scales


def dense(codes, scales, group):
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(1).to(torch.int16)
    c = torch.where(c > 7, c - 16, c).to(F64)
    return c * scales.to(F64).repeat_interleave(group, 1)


def product(x, codes, scales, group):
    """x W^T and the sum of its terms' magnitudes."""
    W = dense(codes, scales, group)
    x = x.to(F64)
    return x @ W.t(), x.abs() @ W.abs().t()


def bound(k):
    # k products summed in fp32 in some order, each addition off by one step at most, and one more for the scale
    return (k + 8) * 2.0 ** -23


SIZES = [
    # m, n_out, k_in, group
    (1, 1, 32, 32), (1, 16, 128, 128), (2, 17, 96, 32), (3, 100, 64, 64), (1, 300, 320, 64), (8, 64, 384, 128),
    (9, 33, 160, 32), (16, 48, 1024, 64), (17, 130, 896, 128), (32, 255, 672, 32), (33, 40, 256, 64),
    (70, 31, 256, 128), (1, 64, 4096, 32), (5, 1000, 2048, 128), (31, 16, 11008, 64),
]


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("size", SIZES, ids=[str(s) for s in SIZES])
def test_linear(size, dt):
    import rank_latent_kv_lk_b200 as lk
    m, n, k, group = size
    g = torch.Generator().manual_seed(n + k)
    codes, scales = weights(n, k, group, g)
    x = torch.randn(m, k, generator=g).to(dt)
    res = torch.randn(m, n, generator=g).to(dt)
    w = lk.W4Weight(codes.cuda(), scales.cuda())
    want, mag = product(x, codes, scales, group)
    tol = bound(k) * mag + 1e-30
    check(lk.w4_linear(w, x.cuda(), y_dtype=F32), want, tol, "fp32")
    check(lk.w4_linear(w, x.cuda()), want, tol + HALF_STEP[dt] * (want.abs() + tol) + 2.0 ** -25, "16 bits")
    both = want + res.to(F64)
    check(lk.w4_linear(w, x.cuda(), residual=res.cuda()), both,
          tol + (HALF_STEP[dt] + 2.0 ** -24) * (both.abs() + tol) + 2.0 ** -25, "residual")


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("size", SIZES, ids=[str(s) for s in SIZES])
def test_swiglu(size, dt):
    import rank_latent_kv_lk_b200 as lk
    m, n, k, group = size
    g = torch.Generator().manual_seed(n + k + 1)
    ga, up = weights(n, k, group, g), weights(n, k, group, g)
    x = torch.randn(m, k, generator=g).to(dt)
    w = lk.W4Weight(ga[0].cuda(), ga[1].cuda(), up[0].cuda(), up[1].cuda())
    a, am = product(x, *ga, group)
    b, bm = product(x, *up, group)
    want = a * torch.sigmoid(a) * b
    # |silu'| <= 1.1; the activation's own exp, division and products: 8 steps
    da, db = bound(k) * am, bound(k) * bm
    tol = 1.1 * da * (b.abs() + db) + (a * torch.sigmoid(a)).abs() * db + 8 * 2.0 ** -23 * want.abs() + 1e-30
    check(lk.w4_linear(w, x.cuda(), y_dtype=F32), want, tol, "fp32")
    check(lk.w4_linear(w, x.cuda()), want, tol + HALF_STEP[dt] * (want.abs() + tol) + 2.0 ** -25, "16 bits")


def test_strided_rows_and_residual_in_place():
    import rank_latent_kv_lk_b200 as lk
    g = torch.Generator().manual_seed(0)
    codes, scales = weights(80, 256, 64, g)
    w = lk.W4Weight(codes.cuda(), scales.cuda())
    wide = torch.randn(6, 512, generator=g).to(BF).cuda()
    x = wide[:, 128:384]
    y = torch.randn(6, 80, generator=g).to(BF).cuda()
    want = lk.w4_linear(w, x.contiguous(), residual=y.clone())
    out = lk.w4_linear(w, x, residual=y, y=y)
    assert out.data_ptr() == y.data_ptr() and torch.equal(out, want)


def test_no_rows():
    import rank_latent_kv_lk_b200 as lk
    g = torch.Generator().manual_seed(0)
    codes, scales = weights(16, 64, 32, g)
    w = lk.W4Weight(codes.cuda(), scales.cuda())
    assert lk.w4_linear(w, torch.empty(0, 64, dtype=BF, device="cuda")).shape == (0, 16)


def test_infinities_stay_in_their_row():
    import rank_latent_kv_lk_b200 as lk
    g = torch.Generator().manual_seed(0)
    codes, scales = weights(40, 128, 128, g)
    w = lk.W4Weight(codes.cuda(), scales.cuda())
    x = torch.randn(3, 128, generator=g).to(HF)
    x[1, 5] = float("inf")
    y = lk.w4_linear(w, x.cuda(), y_dtype=F32).cpu()
    want, mag = product(x[[0, 2]], codes, scales, 128)
    check(y[[0, 2]], want, bound(128) * mag + 1e-30, "other rows")
    assert not torch.isfinite(y[1][dense(codes, scales, 128)[:, 5] != 0]).any()


# More tiles of 16 outputs than the GPU has SMs (148): several a CTA, whose warps share the staged rows of x.  The tiles
# are no multiple of a CTA's in most, the outputs no multiple of 16, the inputs end inside a step of 128, and the steps
# go round the ring or are fewer than its stages.
WIDE = [(2400, 160, 32), (2369, 64, 64), (4090, 192, 64), (4096, 1184, 32), (7000, 384, 128), (9473, 288, 32),
        (11003, 320, 64), (11008, 896, 128), (20001, 160, 32)]


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("m", [1, 5, 16, 32, 33])
@pytest.mark.parametrize("size", WIDE, ids=[str(s) for s in WIDE])
def test_several_tiles_a_cta(size, m, dt):
    import rank_latent_kv_lk_b200 as lk
    n, k, group = size
    g = torch.Generator().manual_seed(n + m)
    one, two = weights(n, k, group, g), weights(n, k, group, g)
    x = torch.randn(m, k, generator=g).to(dt)
    a, am = product(x, *one, group)
    b, bm = product(x, *two, group)
    da, db = bound(k) * am, bound(k) * bm
    w = lk.W4Weight(one[0].cuda(), one[1].cuda())
    check(lk.w4_linear(w, x.cuda(), y_dtype=F32), a, da + 1e-30, "linear")
    res = torch.randn(m, n, generator=g).to(dt)
    both = a + res.to(F64)
    check(lk.w4_linear(w, x.cuda(), residual=res.cuda()), both,
          da + (HALF_STEP[dt] + 2.0 ** -24) * (both.abs() + da) + 2.0 ** -25, "residual")
    w = lk.W4Weight(one[0].cuda(), one[1].cuda(), two[0].cuda(), two[1].cuda())
    want = a * torch.sigmoid(a) * b
    tol = 1.1 * da * (b.abs() + db) + (a * torch.sigmoid(a)).abs() * db + 8 * 2.0 ** -23 * want.abs() + 1e-30
    got = lk.w4_linear(w, x.cuda(), y_dtype=F32)
    check(got, want, tol, "gated")
    for _ in range(5):
        assert torch.equal(lk.w4_linear(w, x.cuda(), y_dtype=F32), got)
