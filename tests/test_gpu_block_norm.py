"""The norms around a block against float64."""
import pytest
import torch

from tests.paged_reference import F64, HALF_STEP

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5


def reference(y, x, w_post, gate, scale, w_pre, eps):
    y, x = y.to(F64), x.to(F64)
    if w_post is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w_post.to(F64)
    if gate is not None:
        y = y * gate.to(F64)
    add = scale * y
    x = x + add
    h = None if w_pre is None else x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w_pre.to(F64)
    return x, h, add


def check(got, want, slack, dt, what):
    got = got.cpu().to(F64)
    tol = slack + HALF_STEP[dt] * (want.abs() + slack) + 2.0 ** -25
    bad = (got - want).abs() - tol
    assert (bad <= 0).all(), f"{what}: over by {float(bad.max()):.3e}"


def run(m, width, dt, post, gate, pre, seed=0, eps=EPS, scale=0.5, offset=0):
    import rank_latent_kv_lk_b200 as lk
    g = torch.Generator().manual_seed(seed)

    def t(*shape):
        n = 1
        for s in shape:
            n *= s
        return torch.randn(n + offset, generator=g).to(dt)

    def on(v, *shape):
        return None if v is None else v.cuda()[offset:].view(shape)

    y, x = 3 * t(m, width), t(m, width)
    wp = t(width) if post else None
    wq = t(width) if pre else None
    gt = {"none": None, "channel": t(width), "token": t(m, width)}[gate]
    gs = (m, width) if gate == "token" else (width,)
    got_x, got_h = lk.rmsnorm_gate_residual(on(y, m, width), on(x, m, width), w_post=on(wp, width), gate=on(gt, *gs),
                                            scale=scale, w_pre=on(wq, width), eps=eps)

    def host(v, *shape):
        return None if v is None else v[offset:].view(shape)

    X, H, add = reference(host(y, m, width), host(x, m, width), host(wp, width), host(gt, *gs), scale,
                          host(wq, width), eps)
    # a mean of squares in fp32: at most `width` roundings, halved by the root; ten more around it
    rel = (width / 2 + 10) * 2.0 ** -24
    slack = rel * add.abs() + 2.0 ** -24 * X.abs()
    check(got_x, X, slack, dt, "x")
    if pre:
        rms = torch.sqrt((X * X).mean(-1, keepdim=True) + eps)
        w = host(wq, width).to(F64).abs()
        check(got_h, H, w / rms * slack + (rel + slack.square().mean(-1, keepdim=True).sqrt() / rms) * H.abs(), dt, "h")
    else:
        assert got_h is None


@pytest.mark.parametrize("dt", [BF, HF, F32])
@pytest.mark.parametrize("m,width", [(1, 1), (2, 7), (3, 8), (1, 64), (5, 100), (33, 1000), (4, 4096), (2, 5003),
                                     (3, 8192), (2, 20000), (1, 32768), (2, 32767),
                                     (9, 2049), (5, 2062), (300, 4127), (1100, 1001), (260, 6631)])
def test_all_parts(dt, m, width):
    run(m, width, dt, True, "channel", True, seed=width)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("pre", [False, True])
def test_parts(post, gate, pre):
    run(6, 768, BF, post, gate, pre)
    run(6, 771, HF, post, gate, pre)


def test_unaligned_tensors():
    run(4, 256, BF, True, "token", True, offset=1)
    run(4, 256, F32, True, "channel", True, offset=3)


def test_rows_of_zeros_and_eps():
    import rank_latent_kv_lk_b200 as lk
    z = torch.zeros(2, 128, dtype=BF, device="cuda")
    w = torch.ones(128, dtype=BF, device="cuda")
    x, h = lk.rmsnorm_gate_residual(z, z, w_post=w, w_pre=w, eps=1e-6)
    assert (x == 0).all() and (h == 0).all()
    run(3, 64, F32, True, "none", True, eps=0.0, scale=-2.0)


@pytest.mark.parametrize("xo,ho", [("x", "y"), ("y", None), ("x", None)])
def test_in_place(xo, ho):
    import rank_latent_kv_lk_b200 as lk
    g = torch.Generator().manual_seed(1)
    for width in (512, 515):
        y, x, w = (torch.randn(*s, generator=g).to(BF).cuda() for s in ((7, width), (7, width), (width,)))
        want = lk.rmsnorm_gate_residual(y, x, w_post=w, w_pre=w)
        t = dict(x=x.clone(), y=y.clone())
        got = lk.rmsnorm_gate_residual(t["y"], t["x"], w_post=w, w_pre=w, x_out=t[xo], h=t.get(ho))
        assert got[0].data_ptr() == t[xo].data_ptr()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_rows():
    import rank_latent_kv_lk_b200 as lk
    e, w = torch.empty(0, 64, dtype=BF, device="cuda"), torch.ones(64, dtype=BF, device="cuda")
    x, h = lk.rmsnorm_gate_residual(e, e, w_pre=w)
    assert x.shape == h.shape == (0, 64)


def test_nan_and_infinity_stay_in_their_row():
    import rank_latent_kv_lk_b200 as lk
    y, w = torch.ones(3, 64, dtype=HF, device="cuda"), torch.ones(64, dtype=HF, device="cuda")
    y[1, 3] = float("nan")
    x, h = lk.rmsnorm_gate_residual(y, y.nan_to_num(), w_post=w, w_pre=w)
    assert torch.isfinite(h[[0, 2]]).all() and torch.isnan(h[1]).all()


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("dt", [BF, HF, F32])
def test_parts_of_long_rows(dt, post, gate, pre):
    # odd widths in whole vectors, and two vectors a thread (256 rows and more)
    for m, width in ((3, 2049), (2, 4099), (5, 2054), (2, 16387), (300, 4096), (257, 1032)):
        run(m, width, dt, post, gate, pre, seed=m)


@pytest.mark.parametrize("xo,ho", [("x", "y"), ("y", None), ("x", None)])
@pytest.mark.parametrize("m,width", [(7, 2049), (4, 4099), (6, 2054), (300, 4096), (257, 1032), (1100, 1001)])
def test_long_rows_in_place(m, width, xo, ho):
    import rank_latent_kv_lk_b200 as lk
    g = torch.Generator().manual_seed(1)
    for dt in (BF, HF, F32):
        y, x, gate, w = (torch.randn(*s, generator=g).to(dt).cuda() for s in (*[(m, width)] * 3, (width,)))
        want = lk.rmsnorm_gate_residual(y, x, w_post=w, gate=gate, w_pre=w)
        t = dict(x=x.clone(), y=y.clone())
        got = lk.rmsnorm_gate_residual(t["y"], t["x"], w_post=w, gate=gate, w_pre=w, x_out=t[xo], h=t.get(ho))
        assert got[0].data_ptr() == t[xo].data_ptr()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rows_beyond_32_bits_of_elements():
    # The last rows of 2^31 elements and more: what those rows give alone, and float64's with the bounds of run().  (Rows
    # of an odd width start at another element of a vector than a copy of them does, and sum in another order: those
    # are held against float64 only.)
    import rank_latent_kv_lk_b200 as lk
    for width in (32768, 32749):
        m = 2 ** 31 // width + 9
        y, x = (torch.zeros(m, width, dtype=BF, device="cuda") for _ in range(2))
        y[-5:].normal_()
        x[-5:].normal_()
        w = torch.ones(width, dtype=BF, device="cuda")
        one = torch.ones(width, dtype=BF)
        X, H, add = reference(y[-5:].cpu(), x[-5:].cpu(), one, None, 1.0, one, EPS)
        alone = lk.rmsnorm_gate_residual(y[-5:].clone(), x[-5:].clone(), w_post=w, w_pre=w)
        got = lk.rmsnorm_gate_residual(y, x, w_post=w, w_pre=w, x_out=x, h=y)
        if width % 8 == 0:
            assert torch.equal(got[0][-5:], alone[0]) and torch.equal(got[1][-5:], alone[1])
        rel = (width / 2 + 10) * 2.0 ** -24
        slack = rel * add.abs() + 2.0 ** -24 * X.abs()
        check(got[0][-5:], X, slack, BF, "x")
        rms = torch.sqrt((X * X).mean(-1, keepdim=True) + EPS)
        check(got[1][-5:], H, slack / rms + (rel + slack.square().mean(-1, keepdim=True).sqrt() / rms) * H.abs(), BF,
              "h")
        assert (got[0][:-5].view(torch.int16) == 0).all()
        del y, x, got
    torch.cuda.empty_cache()
