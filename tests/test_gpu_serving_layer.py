"""The serving operators run together, as a decoder layer uses them: steps with
append, attention, eviction, 4-bit products and norms, in one stream, captured
into a graph, and beside one another on two streams."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F64 = torch.bfloat16, torch.float64
E, NH, NK, D, I, PAGE, GROUP = 256, 8, 2, 64, 512, 16, 64


def w4(n, k, g):
    return (torch.randint(0, 256, (n, k // 2), generator=g).to(torch.uint8),
            (torch.rand(n, k // GROUP, generator=g) * 0.4 / k ** 0.5 + 0.05 / k ** 0.5).to(torch.float16))


def weights(g, post=True, gate=True):
    w = {"qkv": w4((NH + 2 * NK) * D, E, g), "o": w4(E, NH * D, g), "gate": w4(I, E, g), "up": w4(I, E, g),
         "down": w4(E, I, g)}
    for n in ("norm_ffn", "norm_next") + (("post_attn", "post_ffn") if post else ()):
        w[n] = (1 + 0.2 * torch.randn(E, generator=g)).to(BF)
    for n in ("gate_attn", "gate_ffn") if gate else ():
        w[n] = torch.rand(E, generator=g).to(BF)
    return w


def dense(cs):
    codes, scales = cs
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(1).to(torch.int16)
    return torch.where(c > 7, c - 16, c).to(F64) * scales.to(F64).repeat_interleave(GROUP, 1)


class Plain:
    """The layer in float64, K and V per sequence as lists of rows, eviction per head."""

    def __init__(self, w, batch):
        self.W = {k: dense(v) for k, v in w.items() if isinstance(v, tuple)}
        self.n = {k: v.to(F64) for k, v in w.items() if not isinstance(v, tuple)}
        empty = torch.zeros(0, D, dtype=F64)
        self.rows = [[dict(k=empty, v=empty, mass=empty[:, 0], pos=empty[:, 0]) for _ in range(NK)]
                     for _ in range(batch)]
        self.next = [0] * batch

    @staticmethod
    def rms(x):
        return x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5)

    def block(self, y, x, post, gate, pre):
        if post in self.n:
            y = self.rms(y) * self.n[post]
        if gate in self.n:
            y = y * self.n[gate]
        x = x + y
        return x, self.rms(x) * self.n[pre]

    def step(self, x, h):
        qkv = h @ self.W["qkv"].t()
        a = torch.zeros(len(x), NH * D, dtype=F64)
        for b in range(len(x)):
            for j in range(NK):
                r = self.rows[b][j]
                k = qkv[b, (NH + j) * D:(NH + j + 1) * D].to(BF).to(F64)
                v = qkv[b, (NH + NK + j) * D:(NH + NK + j + 1) * D].to(BF).to(F64)
                r["k"], r["v"] = torch.cat((r["k"], k[None])), torch.cat((r["v"], v[None]))
                r["mass"] = torch.cat((r["mass"], torch.zeros(1, dtype=F64)))
                r["pos"] = torch.cat((r["pos"], torch.tensor([self.next[b]], dtype=F64)))
                for i in range(NH // NK):
                    q = qkv[b, (j * (NH // NK) + i) * D:][:D].to(BF).to(F64)
                    p = torch.softmax(r["k"] @ q / D ** 0.5, 0)
                    a[b, (j * (NH // NK) + i) * D:][:D] = p @ r["v"]
                    r["mass"] = r["mass"] + p
            self.next[b] += 1
        x, h = self.block(a @ self.W["o"].t(), x, "post_attn", "gate_attn", "norm_ffn")
        g = h @ self.W["gate"].t()
        y = (g * torch.sigmoid(g) * (h @ self.W["up"].t())) @ self.W["down"].t()
        return self.block(y, x, "post_ffn", "gate_ffn", "norm_next")

    def evict(self, budget, window, n_sink):
        from tests.paged_reference import evict
        for b, heads in enumerate(self.rows):
            for r in heads:
                src = evict(r["mass"].numpy(), r["pos"].numpy(), len(r["pos"]), self.next[b], budget, window, n_sink)
                for n in r:
                    r[n] = r[n][torch.from_numpy(src)]


def setup(batch, mass, seed=0, **kw):
    from rank_latent_kv_lk_b200.layer import W4PagedDecoderLayer
    g = torch.Generator().manual_seed(seed)
    w = weights(g, **kw)
    width = 6
    layer = W4PagedDecoderLayer(w, NH, NK, D, batch * width, PAGE, mass=mass)
    table = torch.randperm(batch * width, generator=g).to(torch.int32).view(batch, width).cuda()
    seq = torch.zeros(batch, dtype=torch.int32, device="cuda")
    xs = [torch.randn(batch, E, generator=g).to(BF) for _ in range(40)]
    return layer, w, table, seq, seq.clone() if mass else None, xs


def first_norm(x):
    import rank_latent_kv_lk_b200 as lk
    one = torch.ones(E, dtype=BF, device="cuda")
    return lk.rmsnorm_gate_residual(torch.zeros_like(x), x, w_pre=one)[1]


@pytest.mark.parametrize("post,gate", [(True, True), (False, False), (True, False)])
def test_steps_against_float64(post, gate):
    # Each of the eight bf16 results of a step is off by at most 2^-8 of its value and its inputs' errors pass on with
    # a gain of order one (norms, softmax averages, residual); 2-norm errors of random signs add as squares: below
    # 2^-8 sqrt(8) in most steps, bounded here by 8 * 2^-8.
    layer, w, table, seq, _, xs = setup(3, False, post=post, gate=gate)
    plain = Plain(w, 3)
    for t in range(12):
        x = xs[t].cuda()
        h = first_norm(x)
        got = layer.step(x, h, table, seq, t + 1)
        want = plain.step(xs[t].to(F64), h.cpu().to(F64))
        for a, b in zip(got, want):
            err = (a.cpu().to(F64) - b).norm() / b.norm()
            assert err <= 8 * 2.0 ** -8, (t, float(err))
    assert seq.tolist() == [12] * 3


def test_steps_with_eviction_keep_the_wanted_tokens():
    import rank_latent_kv_lk_b200 as lk
    layer, w, table, seq, nxt, xs = setup(2, True, seed=3)
    plain = Plain(w, 2)
    for t in range(40):
        x = xs[t].cuda()
        h = first_norm(x)
        got = layer.step(x, h, table, seq, 32, nxt)
        want = plain.step(xs[t].to(F64), h.cpu().to(F64))
        # the plain layer's own weights and order decide; the kernels' order can differ where weights nearly tie, so the
        # plain layer takes the kernels' kept positions over and checks that they are as wanted as its own
        if seq[0].item() >= 24:
            before = [[r["mass"].clone() for r in heads] for heads in plain.rows]
            pos_before = [[r["pos"].clone() for r in heads] for heads in plain.rows]
            layer.evict(table, seq, nxt, 32, 16, window=4, n_sink=2)
            assert seq.tolist() == [16, 16]
            for b in range(2):
                ids = table[b].long().cpu()
                for j in range(NK):
                    pos = layer.cache.pos.cpu()[ids, j].flatten()[:16]
                    assert len(set(pos.tolist())) == 16
                    m, p = before[b][j], pos_before[b][j]
                    keep = torch.isin(p, pos.to(F64))
                    assert int(keep.sum()) == 16
                    safe = (p < 2) | (p >= plain.next[b] - 4)
                    assert keep[safe].all()
                    if (~keep).any() and (keep & ~safe).any():
                        # weights summed over 24 steps of bf16 inputs: a few per cent apart at most
                        assert m[keep & ~safe].min() >= m[~keep].max() * 0.9
                    r = plain.rows[b][j]
                    order = torch.stack([(p == x).nonzero()[0, 0] for x in pos.to(F64)])
                    for n in r:
                        r[n] = r[n][order]
        for a, b in zip(got, want):
            assert (a.cpu().to(F64) - b).norm() / b.norm() <= 8 * 2.0 ** -8, t
    assert nxt.tolist() == [40, 40]
    lk.device_status()


def test_a_captured_step_replays():
    layer, w, table, seq, nxt, xs = setup(2, True, seed=5)
    other, _, table2, seq2, nxt2, _ = setup(2, True, seed=5)
    x, h = xs[0].cuda(), first_norm(xs[0].cuda())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # a first run outside the capture
        layer.step(x, h, table, seq, 64, nxt)
    torch.cuda.current_stream().wait_stream(side)
    other.step(x, h, table2, seq2, 64, nxt2)
    graph = torch.cuda.CUDAGraph()
    sx, sh = x.clone(), h.clone()
    with torch.cuda.graph(graph):
        out = layer.step(sx, sh, table, seq, 64, nxt)
        layer.evict(table, seq, nxt, 64, 8, window=2, n_sink=1)
    for t in range(1, 25):
        x = xs[t].cuda()
        sx.copy_(x)
        sh.copy_(first_norm(x))
        graph.replay()
        want = other.step(x, first_norm(x), table2, seq2, 64, nxt2)
        other.evict(table2, seq2, nxt2, 64, 8, window=2, n_sink=1)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), t
        assert seq.tolist() == seq2.tolist() == [min(t + 1, 8)] * 2
    assert torch.equal(layer.cache.mass, other.cache.mass) and torch.equal(layer.cache.k, other.cache.k)


def test_two_graphs_and_two_streams_share_no_scratch():
    import rank_latent_kv_lk_b200 as lk
    from tests.paged_reference import Pages
    made = []
    for seed in range(2):
        pages = Pages([3000, 700], 2, 128, 16, BF, seed=seed, mass=True)
        q = torch.randn(2, 8, 128, generator=pages.g).to(BF).cuda()
        made.append([pages, pages.cuda(), pages.table.cuda(), pages.seq(), q])
    want = [lk.paged_decode_attn(c, t, q, s, 3000) for _, c, t, s, q in made]
    graphs = []
    for _, c, t, s, q in made:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = lk.paged_decode_attn(c, t, q, s, 3000)
        graphs.append((g, out))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):  # replays and eager calls at the same time
        eager = []
        for (g, _), s, (_, c, t, sl, q) in zip(graphs, streams, made):
            with torch.cuda.stream(s):
                g.replay()
                eager.append(lk.paged_decode_attn(c, t, q, sl, 3000))
        torch.cuda.synchronize()
        for (_, out), e, w in zip(graphs, eager, want):
            assert torch.equal(out, w) and torch.equal(e, w)
    # the `stream` argument is the same as a current stream
    _, c, t, sl, q = made[0]
    got = lk.paged_decode_attn(c, t, q, sl, 3000, stream=streams[1])
    streams[1].synchronize()
    assert torch.equal(got, want[0])


def test_wrappers_refuse_wrong_tensors():
    import rank_latent_kv_lk_b200 as lk
    cache = lk.PagedKVCache(8, 16, 2, 64, mass=True)
    table = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    seq = torch.zeros(2, dtype=torch.int32, device="cuda")
    q = torch.zeros(2, 4, 64, dtype=BF, device="cuda")
    k = torch.zeros(2, 1, 2, 64, dtype=BF, device="cuda")
    lk.paged_decode_attn(cache, table, q, seq, 64)
    for bad in (dict(q=q.cpu()), dict(q=q[..., :32]), dict(q=q.transpose(0, 1)), dict(table=table.long()),
                dict(table=table[:1]), dict(table=table.t().contiguous().t()), dict(seq=seq.long()), dict(seq=seq[:1])):
        a = dict(dict(q=q, table=table, seq=seq), **bad)
        with pytest.raises((ValueError, TypeError)):
            lk.paged_decode_attn(cache, a["table"], a["q"], a["seq"], 64)
    with pytest.raises(TypeError):
        lk.paged_decode_attn(cache, table, q.float(), seq, 64)
    with pytest.raises(lk.LkError):
        lk.paged_decode_attn(cache, table, q, seq, 65)
    with pytest.raises(lk.LkError):
        lk.paged_decode_attn(cache, table, q[:, :3].contiguous(), seq, 64)
    with pytest.raises(ValueError):
        lk.paged_decode_attn(cache, table, q, seq, 64, out=torch.empty(2, 4, 65, device="cuda"))
    for bad in (k[:, :, :1], k.transpose(2, 3).contiguous().transpose(2, 3), k.cpu()):
        with pytest.raises(ValueError):
            lk.paged_append(cache, table, bad, bad, seq, seq)
    with pytest.raises(lk.LkError):
        lk.paged_append(cache, table, k, k, seq)  # a cache with mass needs positions
    with pytest.raises(ValueError):
        lk.paged_evict(lk.PagedKVCache(8, 16, 2, 64), table, seq, seq, 64, 8)
    with pytest.raises(ValueError):
        lk.paged_evict(cache, table, seq, seq, 64, 8, mass_out=torch.empty(3, device="cuda"), pos_out=cache.pos)
    with pytest.raises(TypeError):
        lk.PagedKVCache.from_tensors(cache.k.float(), cache.v.float())
    with pytest.raises(ValueError):
        lk.PagedKVCache.from_tensors(cache.k, cache.v[:4])
    with pytest.raises(ValueError):
        lk.PagedKVCache.from_tensors(cache.k, cache.v, mass=cache.mass)
    codes, scales = w4(32, 128, torch.Generator().manual_seed(0))
    w = lk.W4Weight(codes.cuda(), scales.cuda())
    x = torch.zeros(3, 128, dtype=BF, device="cuda")
    for bad in (x[:, :64], x.t(), x.cpu(), x[0]):
        with pytest.raises(ValueError):
            lk.w4_linear(w, bad)
    with pytest.raises(TypeError):
        lk.w4_linear(w, x.float())
    with pytest.raises((ValueError, TypeError)):
        lk.w4_linear(w, x, residual=torch.zeros(3, 32, device="cuda"))
    with pytest.raises(ValueError):
        lk.W4Weight(codes.cuda(), scales.cuda()[:, :1].expand(32, 3).contiguous())
    y = torch.zeros(3, 64, dtype=BF, device="cuda")
    for bad in (dict(x=y[:2]), dict(gate=y[:, 0]), dict(w_post=y), dict(h=y.clone()), dict(x=y.half())):
        with pytest.raises((ValueError, TypeError)):
            lk.rmsnorm_gate_residual(**dict(dict(y=y, x=y), **bad))
    with pytest.raises(ValueError):
        lk.rmsnorm_gate_residual(y.t(), y.t())


@pytest.mark.parametrize("op", ["attention", "product", "norm"])
def test_memory_of_a_call_on_another_stream(op):
    # The input is freed, and its memory asked for again, while the call still waits on its stream; then the result,
    # while the caller's stream still waits to read it.
    import rank_latent_kv_lk_b200 as lk
    g = torch.Generator().manual_seed(2)
    if op == "attention":
        cache = lk.PagedKVCache.from_tensors(*torch.randn(2, 8, 4, 16, 64, generator=g).to(BF).cuda())
        table = torch.arange(8, dtype=torch.int32, device="cuda").expand(64, 8).contiguous()
        seq = torch.full((64,), 128, dtype=torch.int32, device="cuda")
        x = torch.randn(64, 32, 64, generator=g).to(BF).cuda()

        def call(x, stream=None):
            return lk.paged_decode_attn(cache, table, x, seq, 128, stream=stream)
    elif op == "product":
        w = lk.W4Weight(*(t.cuda() for t in w4(4096, 4096, g)))
        x = torch.randn(32, 4096, generator=g).to(BF).cuda()

        def call(x, stream=None):
            return lk.w4_linear(w, x, stream=stream)
    else:
        x = torch.randn(32, 4096, generator=g).to(BF).cuda()
        one = torch.ones(4096, dtype=BF, device="cuda")

        def call(x, stream=None):
            return lk.rmsnorm_gate_residual(x, x, w_pre=one, stream=stream)[1]
    neg = -2 * x
    want, other = call(x), call(neg)
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    mine = x.clone()
    side.wait_stream(here)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = call(mine, stream=side)
    del mine
    new = [torch.full_like(x, 7) for _ in range(4)]
    here.wait_stream(side)
    torch.cuda._sleep(20_000_000)
    seen = got.clone()
    del got
    more = [call(neg, stream=side) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(seen, want)
    assert all(torch.equal(m, other) for m in more)
    assert all((n == 7).all() for n in new)


def test_no_sequences():
    # as products and norms of no rows: an empty result, and nothing done
    import rank_latent_kv_lk_b200 as lk
    layer, _, _, _, _, _ = setup(1, True)
    before = [t.clone() for t in (layer.cache.k, layer.cache.mass)]
    table = torch.empty(0, 6, dtype=torch.int32, device="cuda")
    n = torch.empty(0, dtype=torch.int32, device="cuda")
    x = torch.empty(0, E, dtype=BF, device="cuda")
    launches = lk.kernel_launches()
    out = layer.step(x, x, table, n, 64, n.clone())
    layer.evict(table, n, n.clone(), 64, 8)
    assert out[0].shape == out[1].shape == (0, E) and lk.kernel_launches() == launches
    q = torch.empty(0, NH, D, dtype=BF, device="cuda")
    assert lk.paged_decode_attn(layer.cache, table, q, n, 64, out_dtype=torch.float32).shape == (0, NH, D)
    with pytest.raises(ValueError):
        lk.paged_decode_attn(layer.cache, table, q[:, :, :16], n, 64)
    assert torch.equal(before[0], layer.cache.k) and torch.equal(before[1], layer.cache.mass)


def test_a_refused_length_allocates_nothing():
    # scratch for 2^24 slots would be gigabytes
    import rank_latent_kv_lk_b200 as lk
    cache = lk.PagedKVCache(8, 16, 2, 64, mass=True)
    table = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    seq = torch.zeros(2, dtype=torch.int32, device="cuda")
    q = torch.zeros(2, 4, 64, dtype=BF, device="cuda")
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    for call in (lambda n: lk.paged_decode_attn(cache, table, q, seq, n, accumulate=True),
                 lambda n: lk.paged_evict(cache, table, seq, seq.clone(), n, 8)):
        for n in (65, 1 << 24, 2 ** 31 - 1):
            with pytest.raises(lk.LkError):
                call(n)
        with pytest.raises(ValueError):
            call(1 << 31)
    assert torch.cuda.max_memory_allocated() - before < 1 << 20


def test_a_side_stream_inside_a_capture():
    # stream= on a stream that forks from the captured one and joins it again
    import rank_latent_kv_lk_b200 as lk
    g = torch.Generator().manual_seed(4)
    w = lk.W4Weight(*(t.cuda() for t in w4(512, 256, g)))
    x, one = torch.randn(4, 256, generator=g).to(BF).cuda(), torch.ones(512, dtype=BF, device="cuda")

    def both(x, side, here):
        y = x + 1
        side.wait_stream(here)
        a = lk.w4_linear(w, y, stream=side)
        del y
        b = lk.w4_linear(w, x)
        here.wait_stream(side)
        return lk.rmsnorm_gate_residual(a, b, w_pre=one)

    here = torch.cuda.current_stream()
    both(x, torch.cuda.Stream(), here)
    graph, sx = torch.cuda.CUDAGraph(), x.clone()
    with torch.cuda.graph(graph):
        out = both(sx, torch.cuda.Stream(), torch.cuda.current_stream())
    for scale in (1.0, -2.0, 0.5):
        sx.copy_(x * scale)
        graph.replay()
        want = both(x * scale, torch.cuda.Stream(), here)
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
