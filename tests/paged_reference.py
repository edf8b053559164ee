"""Plain float64 forms of the paged-cache operators, sequence by sequence and
head by head, and the inputs their tests share."""
import math

import numpy as np
import torch

F64 = torch.float64
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


class Pages:
    """Pools and page tables of sequences of the given lengths.  Every row that
    belongs to no token holds NaN (int8: code 77 with a NaN scale), every table
    entry behind a sequence's last page lies outside the pool."""

    def __init__(self, lens, kv_heads, dim, page, dtype, seed=0, mass=False, extra=0, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.kv_heads, self.dim, self.dtype = list(lens), page, kv_heads, dim, dtype
        need = [-(-(n + extra) // page) for n in lens]
        self.width = max(1, max(need))
        self.n_pages = sum(need) + 3
        perm = torch.randperm(self.n_pages, generator=g).tolist()
        self.table = torch.full((len(lens), self.width), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
            at += n
        shape = (self.n_pages, kv_heads, page, dim)
        live = torch.zeros(shape[:3], dtype=torch.bool)
        for b in range(len(lens)):
            for t in range(lens[b]):
                live[self.table[b, t // page], :, t % page] = True
        self.live = live
        k = torch.randn(shape, generator=g) * spread
        v = torch.randn(shape, generator=g)
        self.k_scale = self.v_scale = self.mass = self.pos = None
        if dtype is torch.int8:
            self.k_scale, self.v_scale = k.abs().amax(-1) / 127, v.abs().amax(-1) / 127 * torch.exp(
                3 * torch.randn(shape[:3], generator=g))
            self.k = torch.round(k / self.k_scale[..., None]).to(torch.int8)
            self.v = torch.round(v / (v.abs().amax(-1) / 127)[..., None]).to(torch.int8)
            for x, s in ((self.k, self.k_scale), (self.v, self.v_scale)):
                x[~live] = 77
                s[~live] = math.nan
        else:
            self.k, self.v = k.to(dtype), v.to(dtype)
            self.k[~live] = math.nan
            self.v[~live] = math.nan
        if mass:
            self.mass = torch.rand(shape[:3], generator=g)
            self.mass[~live] = math.nan
            self.pos = torch.zeros(shape[:3], dtype=torch.int32)
            for b in range(len(lens)):
                for t in range(lens[b]):
                    self.pos[self.table[b, t // page], :, t % page] = t
        self.g = g

    def cuda(self):
        import rank_latent_kv_lk_b200 as lk
        c = [None if t is None else t.cuda() for t in (self.k, self.v, self.k_scale, self.v_scale, self.mass, self.pos)]
        return lk.PagedKVCache.from_tensors(*c)

    def seq(self):
        return torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def rows(self, pool, b, h, n=None):
        """[n, ...] rows of one sequence and head, in slot order."""
        n = self.lens[b] if n is None else n
        if n == 0:
            return pool[:0, 0, 0]
        ids = self.table[b, :-(-n // self.page)].long()
        return pool[ids, h].flatten(0, 1)[:n]

    def dense(self, b, h):
        k, v = self.rows(self.k, b, h).to(F64), self.rows(self.v, b, h).to(F64)
        if self.k_scale is not None:
            k = k * self.rows(self.k_scale, b, h).to(F64)[:, None]
            v = v * self.rows(self.v_scale, b, h).to(F64)[:, None]
        return k, v


def attention(pages, q, scale, want_mass=False):
    """out, tolerance (before the output's rounding) and mass with its tolerance.

    Errors of a kernel with fp32 sums: a score of D terms is off by at most
    ds = D 2^-23 scale sum |q k| (each addition rounds or truncates once), which
    moves a weight by 2 ds relative (numerator and sum); a weight enters as two
    16-bit terms (2^-16); the T weighted values and the joins are summed in fp32
    (T 2^-23, but no more than 2^-14 for the lengths here).  Terms in fp16 (fp16
    and int8 caches) also have a smallest step of 2^-24, so a weight held 2^10
    times larger is off by up to half of it, 2^-35 of the sum (which is at least
    2^10 as held), however small it is; an int8 weight is held relative to a power of two at most twice the
    largest V scale."""
    B, H, D = q.shape
    group = H // pages.kv_heads
    out, tol = torch.zeros(B, H, D, dtype=F64), torch.zeros(B, H, D, dtype=F64)
    mass = mtol = None
    if want_mass:
        mass = pages.mass.to(F64).clone()
        mtol = 2.0 ** -22 * mass.abs()
    for b in range(B):
        n = pages.lens[b]
        for h in range(H):
            hk = h // group
            if n == 0:
                continue
            k, v = pages.dense(b, hk)
            qh = q[b, h].to(F64)
            s = k @ qh * scale
            p = torch.softmax(s, 0) if torch.isfinite(s.max()) else torch.zeros_like(s)
            ds = float((k.abs() @ qh.abs()).max()) * abs(scale) * D * 2.0 ** -23
            out[b, h] = p @ v
            rel = 2 * ds + 2.0 ** -16 + min(n * 2.0 ** -23, 2.0 ** -14)
            tol[b, h] = rel * (p @ v.abs())
            if pages.k_scale is not None:
                vs = pages.rows(pages.v_scale, b, hk).to(F64)
                tol[b, h] += 2.0 ** -35 * 2 * vs.max() * pages.rows(pages.v, b, hk).to(F64).abs().sum(0)
            elif pages.dtype is torch.float16:
                tol[b, h] += 2.0 ** -35 * v.abs().sum(0)
            if want_mass:
                ids = pages.table[b, :-(-n // pages.page)].long()
                add = torch.zeros(len(ids) * pages.page, dtype=F64)
                add[:n] = p
                add = add.view(len(ids), pages.page)
                mass[ids, hk] += add
                mtol[ids, hk] += (2 * ds + 2.0 ** -18) * add
    return out, tol, mass, mtol


def check(got, want, tol, what):
    got = got.detach().cpu().to(F64)
    assert got.shape == want.shape, what
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bad = (got - want).abs() - tol
    assert (bad <= 0).all(), f"{what}: off by up to {float((got - want).abs().max()):.3e}, worst over by " \
                             f"{float(bad.max()):.3e}, {int((bad > 0).sum())} of {bad.numel()}"


def evict(mass, pos, n, next_pos, budget, window, n_sink):
    """Source slot of every slot below min(n, budget), from a sort (numpy)."""
    mass, pos = np.asarray(mass[:n], np.float64), np.asarray(pos[:n])
    if n <= budget:
        return np.arange(n)
    safe = (pos < n_sink) | (pos >= next_pos - window)
    m = np.where(np.isnan(mass), -np.inf, mass)
    order = sorted(range(n), key=lambda t: (not safe[t], np.isnan(mass[t]), -m[t], t))
    kept = np.zeros(n, bool)
    kept[order[:budget]] = True
    src = np.arange(budget)
    src[~kept[:budget]] = np.nonzero(kept[budget:])[0] + budget
    return src
