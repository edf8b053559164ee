"""The serving operators beside the latent path, as cases to be timed and compared.

Four operators of one decoder-layer step over a paged key-value cache:

* ``attn``   attention of one new token per sequence over the pages of its
             cache, grouped heads, optionally after appending the token and
             with the attention weights accumulated per cached token;
* ``evict``  eviction: the tokens with the least accumulated weight leave and
             the kept rows behind the budget move into the free slots;
* ``w4``     products of a few rows with 4-bit weights under group scales,
             with a residual or with gate, up and SwiGLU in one;
* ``norm``   the norm after a block, its gate and residual scale, and the
             norm before the next block.

With ``own`` false, ``run`` computes them with elementary torch operations in
32 bits; with ``own`` true it calls the library.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
_EPS = 1e-5


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one sequence of a 32-head model at its prompt length plus 128 steps: the call where latency counts
        dict(name="attn one sequence", op="attn", batch=1, kv_heads=32, group=1, dim=128, page=16, len=4224,
             ragged=False, dtype="bf16", mass=False, append=False),
        # sequences of very different lengths, one of them empty, grouped heads, long caches
        dict(name="attn ragged 16k", op="attn", batch=8, kv_heads=8, group=4, dim=128, page=64, len=16384,
             ragged=True, dtype="bf16", mass=False, append=False),
        # int8 pages with a scale per token and head, weights accumulated for a later eviction
        dict(name="attn int8 mass", op="attn", batch=32, kv_heads=8, group=4, dim=128, page=32, len=4096,
             ragged=False, dtype="i8", mass=True, append=False),
        # a whole step of a small-head model with shared keys: append, attend, accumulate; an odd length
        dict(name="attn step fp16", op="attn", batch=16, kv_heads=2, group=8, dim=64, page=16, len=8191,
             ragged=False, dtype="fp16", mass=True, append=True),
        # eviction every 64 steps of a full batch: a few rows move
        dict(name="evict steady", op="evict", batch=32, kv_heads=8, dim=128, page=64, len=2112, budget=2048,
             window=128, sinks=4, ragged=False, scrambled=True, dtype="bf16"),
        # eviction after long prompts: most of the cache leaves
        dict(name="evict prompt", op="evict", batch=8, kv_heads=8, dim=128, page=64, len=16384, budget=4096,
             window=256, sinks=4, ragged=True, scrambled=False, dtype="fp16"),
        # one token through an attention output projection with its residual
        dict(name="w4 one row", op="w4", m=1, n=4096, k=4096, group=128, dtype="bf16", epilogue="residual"),
        # one token through gate, up and SwiGLU, small groups
        dict(name="w4 one row swiglu", op="w4", m=1, n=11008, k=4096, group=32, dtype="fp16", epilogue="swiglu"),
        # a small batch through the down projection
        dict(name="w4 eight rows", op="w4", m=8, n=4096, k=11008, group=64, dtype="bf16", epilogue="residual"),
        # a full batch through gate, up and SwiGLU
        dict(name="w4 full batch swiglu", op="w4", m=32, n=11008, k=4096, group=128, dtype="bf16",
             epilogue="swiglu"),
        # a decode step's rows, gate per channel
        dict(name="norm step", op="norm", rows=32, width=4096, dtype="bf16", gate="channel", post=True, pre=True),
        # a prompt's rows, gate per token and channel
        dict(name="norm prompt", op="norm", rows=4096, width=4096, dtype="fp16", gate="token", post=True, pre=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "evict", "w4", "w4", "norm"])
    if op == "attn":
        c = dict(op=op, batch=_log(rng, 1, 32), kv_heads=rng.choice([1, 2, 4, 8, 16, 32]),
                 group=rng.choice([1, 2, 3, 4, 6, 8, 16]), dim=rng.choice([64, 80, 96, 112, 128, 128, 192, 256]),
                 page=rng.choice([16, 32, 64, 128]), len=_log(rng, 1, 16384), ragged=rng.random() < 0.5,
                 dtype=rng.choice(["bf16", "fp16", "i8"]), mass=rng.random() < 0.5, append=False)
        c["append"] = c["dtype"] != "i8" and rng.random() < 0.4
        while c["kv_heads"] * c["group"] > 128:
            c["kv_heads"] //= 2
        while c["batch"] * c["kv_heads"] * c["len"] * c["dim"] * 4 > 2.0e8:
            c["len"] = c["len"] // 2 + 1
        return c
    if op == "evict":
        n = _log(rng, 8, 16384)
        c = dict(op=op, batch=_log(rng, 1, 32), kv_heads=rng.choice([1, 2, 4, 8, 16, 32]),
                 dim=rng.choice([64, 80, 128, 128, 256]), page=rng.choice([16, 32, 64, 128]), len=n,
                 budget=1, window=0, sinks=0, ragged=rng.random() < 0.5,
                 scrambled=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp16"]))
        while c["batch"] * c["kv_heads"] * c["len"] * c["dim"] * 4 > 2.0e8:
            c["len"] = c["len"] // 2 + 1
        c["budget"] = max(1, min(c["len"], _log(rng, max(1, c["len"] // 8), c["len"])))
        c["window"] = rng.randint(0, c["budget"] // 2)
        c["sinks"] = rng.choice([0, min(4, c["budget"] // 4)])
        return c
    if op == "w4":
        group = rng.choice([32, 64, 128])
        return dict(op=op, m=_log(rng, 1, 32), n=_log(rng, 64, 11008), k=group * max(1, _log(rng, 64, 8192) // group),
                    group=group, dtype=rng.choice(["bf16", "fp16"]),
                    epilogue=rng.choice(["none", "residual", "swiglu"]))
    rows = _log(rng, 1, 4096)
    return dict(op=op, rows=rows, width=_log(rng, 64, min(8192, 16777216 // rows)), dtype=rng.choice(["bf16", "fp16"]),
                gate=rng.choice(["none", "channel", "token"]), post=rng.random() < 0.8, pre=rng.random() < 0.8)


def _lens(case):
    """The sequences' lengths, by the case alone: spread over the range, one full, one empty in larger batches."""
    n, L = case["batch"], case["len"]
    if not case["ragged"]:
        return [L] * n
    lens = [1 + int((L - 1) * (((i + 1) * 0.6180339887) % 1.0)) for i in range(n)]
    if n >= 4:
        lens[1] = 0
    lens[-1] = L
    return lens


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)


def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _prepare_pages(case, g, extra):
    """Pools and page tables: a sequence's pages lie anywhere in the pool, in any order."""
    B, page = case["batch"], case["page"]
    lens = _lens(case)
    need = [-(-(n + extra) // page) for n in lens]
    width = max(1, max(need))
    n_pages = sum(need) + 4
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at, host = 0, perm.cpu()
    for b in range(B):
        table[b, :need[b]] = host[at:at + need[b]]
        at += need[b]
    return dict(lens=lens, table=table.cuda(), n_pages=n_pages, spare=int(host[-1]),
                seq_len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                max_len=max(1, max(lens) + extra))


def _prepare_attn(case, g):
    B, Hk, G, D = case["batch"], case["kv_heads"], case["group"], case["dim"]
    s = _prepare_pages(case, g, 1 if case["append"] else 0)
    shape = (s["n_pages"], Hk, case["page"], D)
    base = _randn((Hk, 1, D), g)                      # a direction that queries share: the first tokens draw attention
    q = 1.5 * _randn((B, Hk, G, D), g) + base
    dt = torch.bfloat16 if case["dtype"] == "i8" else _DT[case["dtype"]]
    s["q"] = q.reshape(B, Hk * G, D).to(dt)
    k = torch.empty(shape, dtype=dt, device="cuda")
    v = torch.empty(shape, dtype=dt, device="cuda")
    k.normal_(generator=g)
    v.normal_(generator=g)
    first = s["table"][:, 0].clamp_min(0).long()
    k[first, :, :4] += base.to(dt)
    s["k_scale"] = s["v_scale"] = None
    if case["dtype"] == "i8":
        for name, x in (("k", k), ("v", v)):
            x = x.float()
            sc = x.abs().amax(-1) / torch.full((), 127.0, device="cuda")
            s[name + "_scale"] = sc
            s[name] = torch.round(x / sc[..., None]).clamp_(-127, 127).to(torch.int8)
    else:
        s["k"], s["v"] = k, v
    s["mass"] = s["pos"] = s["next_pos"] = None
    if case["mass"]:
        s["mass"] = torch.rand(shape[:3], generator=g, device="cuda")
        s["pos"] = torch.zeros(shape[:3], dtype=torch.int32, device="cuda")
        s["next_pos"] = s["seq_len"] + 5
    if case["append"]:
        s["k_new"], s["v_new"] = _randn((B, 1, Hk, D), g, dt), _randn((B, 1, Hk, D), g, dt)
        s["seq_out"] = torch.zeros_like(s["seq_len"])
        s["next_out"] = torch.zeros_like(s["seq_len"]) if case["mass"] else None
    if own:
        import rank_latent_kv_lk_b200 as lk
        s["cache"] = lk.PagedKVCache.from_tensors(s["k"], s["v"], s["k_scale"], s["v_scale"], s["mass"], s["pos"])
    return s


def _prepare_evict(case, g):
    Hk, D, page = case["kv_heads"], case["dim"], case["page"]
    s = _prepare_pages(case, g, 0)
    shape = (s["n_pages"], Hk, page, D)
    s["k"] = torch.empty(shape, dtype=_DT[case["dtype"]], device="cuda").normal_(generator=g)
    s["v"] = torch.empty(shape, dtype=_DT[case["dtype"]], device="cuda").normal_(generator=g)
    # accumulated weights spread over decades; tokens no query has looked at tie at zero
    mass = torch.exp(2.0 * _randn(shape[:3], g))
    s["mass"] = torch.where(torch.rand(shape[:3], generator=g, device="cuda") < 0.02, torch.zeros_like(mass), mass)
    s["pos"] = torch.zeros(shape[:3], dtype=torch.int32, device="cuda")
    s["next_pos"] = s["seq_len"] + (1000 if case["scrambled"] else 0)
    for b, n in enumerate(s["lens"]):
        if n:
            pages = s["table"][b, :-(-n // page)].long()
            t = len(pages) * page
            p = torch.arange(t, device="cuda", dtype=torch.int32).repeat(Hk, 1)
            if case["scrambled"]:  # a cache that was evicted from before: slots are not in order of position
                order = torch.rand((Hk, t), generator=g, device="cuda")
                order[:, n:] = 2.0
                p = order.argsort(-1).to(torch.int32) + 1000
            s["pos"][pages] = p.view(Hk, len(pages), page).transpose(0, 1)
    s["mass_out"], s["pos_out"] = torch.zeros_like(s["mass"]), torch.zeros_like(s["pos"])
    s["seq_out"] = torch.zeros_like(s["seq_len"])
    if own:
        import rank_latent_kv_lk_b200 as lk
        s["cache"] = lk.PagedKVCache.from_tensors(s["k"], s["v"], None, None, s["mass"], s["pos"])
    return s


def _prepare_w4(case, g):
    m, n, k, grp = case["m"], case["n"], case["k"], case["group"]
    dt = _DT[case["dtype"]]
    x = _randn((m, k), g)
    x = torch.where(torch.rand(k, generator=g, device="cuda") < 0.01, 10.0 * x, x)  # a few channels stand out
    s = dict(x=x.to(dt), residual=None)
    for name in ("a", "b") if case["epilogue"] == "swiglu" else ("a",):
        lo, hi = torch.randint(-7, 8, (2, n, k // 2), generator=g, device="cuda", dtype=torch.int32)
        s["codes_" + name] = ((lo & 15) | ((hi & 15) << 4)).to(torch.uint8)
        sc = 0.5 + torch.rand((n, k // grp), generator=g, device="cuda")
        s["scales_" + name] = (sc / (4.0 * math.sqrt(k))).to(torch.float16)
    if case["epilogue"] == "residual":
        s["residual"] = _randn((m, n), g, dt)
    if own:
        import rank_latent_kv_lk_b200 as lk
        s["weight"] = lk.W4Weight(s["codes_a"], s["scales_a"], s.get("codes_b"), s.get("scales_b"))
    return s


def _prepare_norm(case, g):
    rows, width, dt = case["rows"], case["width"], _DT[case["dtype"]]
    s = dict(y=_randn((rows, width), g, dt) * 3, x=_randn((rows, width), g, dt), gate=None, w_post=None, w_pre=None)
    if case["gate"] != "none":
        s["gate"] = _randn((width,) if case["gate"] == "channel" else (rows, width), g, dt)
    if case["post"]:
        s["w_post"] = (1 + 0.1 * _randn((width,), g)).to(dt)
    if case["pre"]:
        s["w_pre"] = (1 + 0.1 * _randn((width,), g)).to(dt)
    return s


def prepare(case, seed):
    make = dict(attn=_prepare_attn, evict=_prepare_evict, w4=_prepare_w4, norm=_prepare_norm)[case["op"]]
    s = make(case, _gen(seed))
    s["case"] = case
    return s


# ------------------------------------------------------------------ one pass

def _attn_plain(s):
    case = s["case"]
    B, Hk, G, D, page = case["batch"], case["kv_heads"], case["group"], case["dim"], case["page"]
    k, v, mass, seq = s["k"], s["v"], s["mass"], s["seq_len"]
    pages = torch.where(s["table"] < 0, s["spare"], s["table"]).long()
    if case["append"]:
        at = pages.gather(1, (seq // page).long()[:, None])[:, 0]
        off = (seq % page).long()
        k[at, :, off] = s["k_new"][:, 0]
        v[at, :, off] = s["v_new"][:, 0]
        if mass is not None:
            mass[at, :, off] = 0.0
            s["pos"][at, :, off] = s["next_pos"][:, None].expand(B, Hk)
            s["next_out"].copy_(s["next_pos"] + 1)
        s["seq_out"].copy_(seq + 1)
        seq = s["seq_out"]
    T = pages.shape[1] * page

    def rows(pool, scale):
        x = pool[pages].float()
        if scale is not None:
            x = x * scale[pages][..., None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hk, T, D)

    q = s["q"].float().view(B, Hk, G, D)
    sc = (q @ rows(k, s["k_scale"]).transpose(-1, -2)) * (1.0 / math.sqrt(D))
    live = torch.arange(T, device="cuda") < seq[:, None, None, None]
    sc = sc.masked_fill(~live, -math.inf)
    top = sc.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = torch.exp(sc - top)
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-38)
    out = (p @ rows(v, s["v_scale"])).reshape(B, Hk * G, D).to(s["q"].dtype)
    got = [out]
    if mass is not None:
        add = p.sum(2).view(B, Hk, pages.shape[1], page).transpose(1, 2)
        mass[pages] = mass[pages] + add
        got.append(mass)
    if case["append"]:
        got += [k, v, seq]
    return got


def _attn_own(s):
    import rank_latent_kv_lk_b200 as lk
    case, seq = s["case"], s["seq_len"]
    if case["append"]:
        lk.paged_append(s["cache"], s["table"], s["k_new"], s["v_new"], seq, s["next_pos"], seq_len_out=s["seq_out"],
                        next_pos_out=s["next_out"])
        seq = s["seq_out"]
    got = [lk.paged_decode_attn(s["cache"], s["table"], s["q"], seq, s["max_len"], accumulate=case["mass"])]
    if case["mass"]:
        got.append(s["mass"])
    if case["append"]:
        got += [s["k"], s["v"], seq]
    return got


def _evict_plain(s):
    case = s["case"]
    B, Hk, page, budget = case["batch"], case["kv_heads"], case["page"], case["budget"]
    pages = torch.where(s["table"] < 0, s["spare"], s["table"]).long()
    T = pages.shape[1] * page

    def rows(pool):
        return pool[pages].transpose(1, 2).reshape(B, Hk, T)

    slot = torch.arange(T, device="cuda")
    seq = s["seq_len"][:, None, None]
    mass, pos = rows(s["mass"]), rows(s["pos"])
    safe = (pos < case["sinks"]) | (pos >= s["next_pos"][:, None, None] - case["window"])
    live = slot < seq
    # most wanted first: protected, then by weight, ties by slot; slots behind the sequence last
    order = torch.sort(mass, dim=-1, descending=True, stable=True).indices
    tier = torch.where(live, safe.long(), torch.full_like(order, -1)).gather(-1, order)
    order = order.gather(-1, torch.sort(tier, dim=-1, descending=True, stable=True).indices)
    rank = torch.empty_like(order).scatter_(-1, order, slot.expand_as(order))
    kept = live & (rank < budget)
    N = min(budget, T)
    sources = torch.where(kept & (slot >= budget), slot, T).sort(-1).values
    hole = ~kept[..., :N]
    nth = (hole.long().cumsum(-1) - 1).clamp_min(0)
    src = torch.where(hole, sources.gather(-1, nth), slot[:N])
    written = (slot[:N] < seq).expand(B, Hk, N)
    src = torch.where(written, src, slot[:N])

    # rows behind a short sequence are left as they are: the spare page stands in for both ends of such a move
    head = torch.arange(Hk, device="cuda")[None, :, None].expand(B, Hk, N)
    end = slot[:N].expand(B, Hk, N)
    dst_page = torch.where(written, pages[:, None].expand(B, Hk, -1).gather(-1, end // page), s["spare"])
    src_page = torch.where(written, pages[:, None].expand(B, Hk, -1).gather(-1, src // page), s["spare"])
    d = (dst_page, head, end % page)
    f = (src_page, head, src % page)
    s["k"][d] = s["k"][f]
    s["v"][d] = s["v"][f]
    s["mass_out"][d] = torch.where(written, s["mass"][f], 0.0)
    s["pos_out"][d] = torch.where(written, s["pos"][f], 0)
    s["seq_out"].copy_(s["seq_len"].clamp_max(budget))
    return [s["k"], s["v"], s["mass_out"], s["pos_out"], s["seq_out"]]


def _evict_own(s):
    import rank_latent_kv_lk_b200 as lk
    case = s["case"]
    lk.paged_evict(s["cache"], s["table"], s["seq_len"], s["next_pos"], s["max_len"], case["budget"],
                   window=case["window"], n_sink=case["sinks"], mass_out=s["mass_out"], pos_out=s["pos_out"],
                   seq_len_out=s["seq_out"])
    return [s["k"], s["v"], s["mass_out"], s["pos_out"], s["seq_out"]]


def _w4_dequant(codes, scales, group, dtype):
    c = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(1).to(dtype)
    c = torch.where(c > 7, c - 16, c)
    return c * scales.to(dtype).repeat_interleave(group, dim=1)


def _w4_plain(s):
    case = s["case"]
    x = s["x"].float()
    y = x @ _w4_dequant(s["codes_a"], s["scales_a"], case["group"], torch.float32).t()
    if case["epilogue"] == "swiglu":
        y = y * torch.sigmoid(y) * (x @ _w4_dequant(s["codes_b"], s["scales_b"], case["group"], torch.float32).t())
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["x"].dtype)


def _w4_own(s):
    import rank_latent_kv_lk_b200 as lk
    return lk.w4_linear(s["weight"], s["x"], residual=s["residual"])


_RES_SCALE = 0.5


def _norm_plain(s):
    y, x = s["y"].float(), s["x"].float()
    if s["w_post"] is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + _EPS) * s["w_post"].float()
    if s["gate"] is not None:
        y = y * s["gate"].float()
    x = x + _RES_SCALE * y
    got = [x.to(s["x"].dtype)]
    if s["w_pre"] is not None:
        got.append((x / torch.sqrt((x * x).mean(-1, keepdim=True) + _EPS) * s["w_pre"].float()).to(s["x"].dtype))
    return got


def _norm_own(s):
    import rank_latent_kv_lk_b200 as lk
    x, h = lk.rmsnorm_gate_residual(s["y"], s["x"], w_post=s["w_post"], gate=s["gate"], scale=_RES_SCALE,
                                    w_pre=s["w_pre"], eps=_EPS)
    return [x] if h is None else [x, h]


def run(state):
    plain = dict(attn=_attn_plain, evict=_evict_plain, w4=_w4_plain, norm=_norm_plain)
    mine = dict(attn=_attn_own, evict=_evict_own, w4=_w4_own, norm=_norm_own)
    return (mine if own else plain)[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "attn":
        Hk, G, D, B = case["kv_heads"], case["group"], case["dim"], case["batch"]
        es = 1 if case["dtype"] == "i8" else 2
        tokens = sum(_lens(case)) + (B if case["append"] else 0)
        per = 2 * D * es + (8 if es == 1 else 0) + (8 if case["mass"] else 0)
        io = 2 * B * Hk * G * D * 2 + (2 * B * Hk * D * es if case["append"] else 0)
        return {"bytes": tokens * Hk * per + io + 4 * tokens // case["page"], "flops": 4 * tokens * Hk * G * D}
    if case["op"] == "evict":
        by, W = 0.0, case["window"] + case["sinks"]
        for n in _lens(case):
            keep = min(n, case["budget"])
            by += case["kv_heads"] * 8 * (n + keep)
            if n > keep:  # kept rows that lie behind the budget: the newest in order, else by chance
                if case["scrambled"]:
                    moved = keep * (n - keep) / n
                else:
                    w = min(case["window"], n - keep)
                    moved = w + max(0, keep - W) * max(0, n - keep - w) / max(1, n - W)
                by += case["kv_heads"] * moved * 2 * 2 * case["dim"] * 2
        return {"bytes": by, "flops": 0.0}
    if case["op"] == "w4":
        m, n, k = case["m"], case["n"], case["k"]
        mats = 2 if case["epilogue"] == "swiglu" else 1
        io = 2 * m * k + 2 * m * n * (2 if case["epilogue"] == "residual" else 1)
        return {"bytes": mats * (n * k // 2 + 2 * n * k // case["group"]) + io, "flops": 2 * mats * m * n * k}
    n = case["rows"] * case["width"]
    tensors = 3 + (1 if case["pre"] else 0) + (1 if case["gate"] == "token" else 0)
    return {"bytes": 2 * n * tensors + 2 * 3 * case["width"], "flops": 10 * n}


# ------------------------------------------------------------------ the definition in 64 bits

def _attn_exact(s):
    """Sequence by sequence, from the definition, on rows laid out one after another."""
    case = s["case"]
    Hk, G, D, page = case["kv_heads"], case["group"], case["dim"], case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    mass = None if s["mass"] is None else s["mass"].double()
    k, v, lens = s["k"], s["v"], list(s["lens"])
    for b in range(case["batch"]):
        table = s["table"][b].tolist()
        if case["append"]:
            t = lens[b]
            k[table[t // page], :, t % page] = s["k_new"][b, 0]
            v[table[t // page], :, t % page] = s["v_new"][b, 0]
            if mass is not None:
                mass[table[t // page], :, t % page] = 0.0
            lens[b] = t + 1
        if lens[b] == 0:
            continue
        ids = torch.tensor(table[:-(-lens[b] // page)], device="cuda")
        for h in range(Hk):
            kk = k[ids, h].reshape(-1, D)[:lens[b]].double()
            vv = v[ids, h].reshape(-1, D)[:lens[b]].double()
            if s["k_scale"] is not None:
                kk = kk * s["k_scale"][ids, h].reshape(-1, 1)[:lens[b]].double()
                vv = vv * s["v_scale"][ids, h].reshape(-1, 1)[:lens[b]].double()
            w = torch.softmax(s["q"][b, h * G:(h + 1) * G].double() @ kk.t() / math.sqrt(D), dim=-1)
            out[b, h * G:(h + 1) * G] = w @ vv
            if mass is not None:
                add = torch.zeros(len(ids) * page, dtype=torch.float64, device="cuda")
                add[:lens[b]] = w.sum(0)
                mass[ids, h] += add.view(-1, page)
    got = [out] + ([] if mass is None else [mass])
    return got + ([k, v, None] if case["append"] else [])


def _evict_exact(s):
    """Unit by unit: a list of slots ordered by (protected, weight, slot), the first ones kept."""
    case = s["case"]
    page, budget = case["page"], case["budget"]
    mass_out = torch.zeros(s["mass"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"]):
        if n == 0:
            continue
        ids = s["table"][b, :-(-n // page)].long()
        newest = int(s["next_pos"][b]) - case["window"]
        for h in range(case["kv_heads"]):
            w = s["mass"][ids, h].reshape(-1)[:n].double()
            p = s["pos"][ids, h].reshape(-1)[:n]
            w = torch.where((p < case["sinks"]) | (p >= newest), w + 1e300, w)
            # equal weights among the protected stay apart only by slot; they are all kept when they fit
            best = torch.argsort(-w, stable=True)[:budget]
            kept = torch.zeros(n, dtype=torch.bool, device="cuda")
            kept[best] = True
            holes = torch.nonzero(~kept[:min(budget, n)])[:, 0]
            moved = torch.nonzero(kept[budget:])[:, 0] + budget
            for pool in (s["k"], s["v"]):
                pool[ids[holes // page], h, holes % page] = pool[ids[moved // page], h, moved % page]
            m = s["mass"][ids, h].reshape(-1)[:n].double()
            m[holes] = m[moved]
            t = torch.arange(min(budget, n), device="cuda")
            mass_out[ids[t // page], h, t % page] = m[:min(budget, n)]
    return [s["k"], s["v"], mass_out, None, None]


def _w4_exact(s):
    case = s["case"]
    x = s["x"].double()

    def product(codes, scales):
        c = codes.to(torch.int64)
        even, odd = ((c % 16) + 8) % 16 - 8, ((c // 16) + 8) % 16 - 8
        sc = scales.double().repeat_interleave(case["group"] // 2, dim=1)
        return x[:, 0::2] @ (even * sc).t() + x[:, 1::2] @ (odd * sc).t()

    y = product(s["codes_a"], s["scales_a"])
    if case["epilogue"] == "swiglu":
        y = y / (1.0 + torch.exp(-y)) * product(s["codes_b"], s["scales_b"])
    return y if s["residual"] is None else y + s["residual"].double()


def _norm_exact(s):
    z = s["y"].double()
    if s["w_post"] is not None:
        z = s["w_post"].double() * z * torch.rsqrt(z.square().sum(-1, keepdim=True) / z.shape[-1] + _EPS)
    z = z if s["gate"] is None else s["gate"].double() * z
    x = s["x"].double() + z * _RES_SCALE
    if s["w_pre"] is None:
        return [x]
    return [x, s["w_pre"].double() * x * torch.rsqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + _EPS)]


def exact(case, seed):
    """What ``run`` returns, from the definitions in 64 bits."""
    s = prepare(case, seed)
    return dict(attn=_attn_exact, evict=_evict_exact, w4=_w4_exact, norm=_norm_exact)[case["op"]](s)
