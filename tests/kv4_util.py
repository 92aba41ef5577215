"""Plain models in 64 bits of the 4-bit cache format, of attention over it, of accumulated
attention weight and of eviction. Test infrastructure only."""
import math

import torch

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DEV = "cuda"


def i32(a, dev=DEV):
    return torch.tensor(a, dtype=torch.int32, device=dev)


def e4m3_values(dev="cpu"):
    return torch.arange(127, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn).double()


def nearest(x, grid):
    """Index of the entry of the ascending grid nearest to each x >= 0, ties to the even index."""
    hi = torch.searchsorted(grid, x.contiguous()).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    down, up = x - grid[lo], grid[hi] - x
    return torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)


def quantise(x, hs):
    """x [..., d] (any float type) with head scale hs (broadcastable to [..., 1], fp32) ->
    (codes uint8 [..., d / 2], scales uint8 [..., d / 16]). Quotients in 64 bits: with x of 8
    significant bits, hs of 24 and 4 more, a quotient that is not the middle of two codes is
    away from it by 2^-32 of itself or more, so that its rounding to 64 bits decides nothing."""
    b = x.double().unflatten(-1, (-1, 16))
    hs = hs.double().unsqueeze(-1)
    grid = e4m3_values(x.device)
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad[..., None], torch.zeros_like(b), b)
    c = nearest(b.abs().amax(-1) / (6 * hs.squeeze(-1)), grid)
    unit = grid[c][..., None] * hs
    y = torch.where(unit > 0, b.abs() / torch.where(unit > 0, unit, torch.ones_like(unit)),
                    torch.zeros_like(b))
    e = nearest(y, torch.tensor(E2M1, dtype=torch.float64, device=x.device))
    e = (e + 8 * ((b < 0) & (unit > 0))).to(torch.uint8).flatten(-2)
    c = torch.where(bad, torch.full_like(c, 127), c).to(torch.uint8)
    return e[..., 0::2] | (e[..., 1::2] << 4), c


def values(codes, scales, hs):
    """What codes [..., d / 2] with scales uint8 [..., d / 16] stand for, in 64 bits."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=codes.device)
    e = lut[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()]
    u = scales.view(torch.float8_e4m3fn).double() * hs.double()
    return (e.unflatten(-1, (-1, 16)) * u[..., None]).flatten(-2)


def block_table(lens, bs, gen, spare=3, extra=1):
    """(table [B, stride] int32 on the CPU, number of pages), pages placed at random."""
    pages = [-(-n // bs) for n in lens]
    blocks = sum(pages) + spare
    place = torch.randperm(blocks, generator=gen).tolist()
    table = torch.full((len(lens), max(pages + [0]) + extra), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = torch.tensor(place[at:at + n], dtype=torch.int32)
        at += n
    return table, blocks


class Cache:
    """A K/V cache of `kind` ("bf16", "e4m3", "kv4") for sequences of these lengths, every row
    that no sequence owns filled with what reads as NaN."""

    def __init__(self, kind, lens, Hkv, d, bs, seed, dev=DEV, spread=1.0):
        gen = torch.Generator().manual_seed(seed)
        self.kind, self.Hkv, self.d, self.bs, self.lens = kind, Hkv, d, bs, lens
        self.table, self.blocks = block_table(lens, bs, gen)
        own = torch.zeros(self.blocks * bs, dtype=torch.bool)
        for b, n in enumerate(lens):
            own[self.rows(b, n)] = True
        shape = (self.blocks * bs, Hkv)
        self.scales = None
        if kind == "kv4":
            self.hs = (torch.rand(2, Hkv, generator=gen) + 0.5) * spread / 64
            self.k, self.v = (torch.randint(0, 256, (*shape, d // 2), generator=gen, dtype=torch.uint8)
                              for _ in "kv")
            self.scales = torch.randint(8, 96, (*shape, 2, d // 16), generator=gen, dtype=torch.uint8)
            self.scales[~own] = 0x7f
        else:
            self.hs = None if kind == "bf16" else (torch.rand(2, Hkv, generator=gen) + 0.5) * spread
            x = torch.randn(2, *shape, d, generator=gen) * spread
            x[:, ~own] = math.nan
            x = x.to(torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn)
            self.k, self.v = x[0], x[1]
        put = lambda t: None if t is None else t.view(self.blocks, bs, *t.shape[1:]).contiguous().to(dev)  # noqa: E731
        self.k, self.v, self.scales = put(self.k), put(self.v), put(self.scales)
        self.hs = None if self.hs is None else self.hs.to(dev)
        self.host_table, self.table = self.table, self.table.to(dev)

    def rows(self, b, n):
        """Flat cache rows of the first n positions of sequence b."""
        t = self.host_table if hasattr(self, "host_table") else self.table
        j = torch.arange(n)
        return t[b, j // self.bs].long() * self.bs + j % self.bs

    def dense(self, b, n, which):
        """K (0) or V (1) of the first n positions, [n, Hkv, d] in 64 bits."""
        at = self.rows(b, n).to(self.k.device)
        x = (self.k, self.v)[which].flatten(0, 1)[at]
        if self.kind == "kv4":
            return values(x, self.scales.flatten(0, 1)[at][:, :, which], self.hs[which][:, None])
        x = x.double()
        return x if self.hs is None else x * self.hs[which].double()[:, None]


def attention(q, K, V, T, D, G, scale, window=0):
    """One sequence's window rows q [1 + D, Hq, d] over K, V [T + 1 + D, Hkv, d] in 64 bits:
    (weights [Hkv, W, G, n], log-sums [W, Hq], out [W, Hq, d] or None, what bounds the errors:
    per row scale * max_j sum |q k|, and sum_j p_j |v_j|)."""
    W, n, Hkv, d = 1 + D, T + 1 + D, K.shape[1], K.shape[2]
    Q = q.double().view(W, Hkv, G, d).permute(1, 0, 2, 3).reshape(Hkv, W * G, d)
    Kt = K.permute(1, 2, 0)
    S = (Q @ Kt * scale).view(Hkv, W, G, n)
    size = (Q.abs() @ Kt.abs() * scale).view(Hkv, W, G, n)
    j = torch.arange(n, device=q.device)
    i = torch.arange(W, device=q.device)[:, None]
    hide = (j > T + i) | ((j < T + i + 1 - window) if window > 0 else False)
    S = S.masked_fill(hide[None, :, None, :], -math.inf)
    size = size.masked_fill(hide[None, :, None, :], 0.0).amax(-1)
    L = S.logsumexp(-1)
    P = (S - L[..., None]).exp()
    flat = lambda x: x.permute(1, 0, 2).reshape(W, Hkv * G)  # noqa: E731
    out = spread = None
    if V is not None:
        Pm = P.reshape(Hkv, W * G, n)
        o2 = lambda x: (Pm @ x.permute(1, 0, 2)).view(Hkv, W, G, d).permute(1, 0, 2, 3).reshape(W, Hkv * G, d)  # noqa: E731
        # A weight is held in f16 before P V: besides 2^-11 of itself, below 2^-14 it is off by up
        # to half of f16's least step, 2^-25, where the row's largest is 2^7 or more and with it
        # the normaliser: 2^-32 of |v_j| for each key, 2^-11 times what is added here.
        out, spread = o2(V), o2(V.abs()) + V.abs().sum(0).repeat_interleave(G, 0) * 2 ** -21
    return P, flat(L), out, flat(size), spread


def evict(mass, n, m, first, last):
    """The positions that one head keeps, in order; mass: a list."""
    if m == n:
        return list(range(n))
    sure = set(range(first)) | set(range(n - last, n))
    w = [-math.inf if math.isnan(x) else x for x in mass]
    nan = [math.isnan(x) for x in mass]
    rest = sorted((j for j in range(n) if j not in sure), key=lambda j: (nan[j], -w[j], j))
    return sorted(sure | set(rest[:m - len(sure)]))
