"""Shared by the tests of rotary positions and of the paged cache: caches with shuffled
pages, and the operators' definitions in 64 bits."""
import math

import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half a step


def int32(x, dev="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def starts(lengths):
    return [sum(lengths[:b]) for b in range(len(lengths) + 1)]


class Cache:
    """Pages of keys and values whose slots beyond the rows' keys, and whose pages that no row
    owns, hold NaN; table entries past a row's keys name no page.  layout: the order of the
    dimensions in memory ("psh", "phs", "hps", "kv": keys and values of a page next to each
    other)."""

    def __init__(self, lens, Hk, d, page, dtype, seed=0, layout="psh", dev="cuda", extra=3, fill=True):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Hk, self.d, self.page, self.dtype = [max(0, n) for n in lens], Hk, d, page, dtype
        need = [-(-n // page) for n in self.lens]
        pages, width = sum(need) + extra, max(need + [0]) + 2
        order = torch.randperm(pages, generator=g).tolist()
        table = torch.full((len(lens), width), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.host_table = table
        self.table = table.to(dev)
        shape = dict(p=pages, s=page, h=Hk)
        if layout == "kv":
            both = torch.full((pages, 2, page, Hk, d), math.nan, dtype=dtype, device=dev)
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            def pool():
                t = torch.full((*(shape[c] for c in layout), d), math.nan, dtype=dtype, device=dev)
                return t.permute(*(layout.index(c) for c in "psh"), 3)
            self.k, self.v = pool(), pool()
        self.rows = []  # keys and values [n, Hk, d] of each row
        for b, n in enumerate(self.lens):
            k, v = (torch.randn(n, Hk, d, generator=g).to(dtype).to(dev) for _ in range(2))
            self.rows.append((k, v))
            if fill:
                self.put(b, 0, k, v)

    def places(self, b, lo, hi):
        j = torch.arange(lo, hi)
        return self.host_table[b].long()[j // self.page].to(self.k.device), (j % self.page).to(self.k.device)

    def put(self, b, lo, k, v):
        if k.shape[0]:
            p, s = self.places(b, lo, lo + k.shape[0])
            self.k[p, s] = k
            self.v[p, s] = v

    def get(self, b, lo, hi):
        p, s = self.places(b, lo, hi)
        return self.k[p, s], self.v[p, s]


def turn(x, pos, f, axes=None, pairs=False, inverse=False):
    """Rotation in 64 bits: x [N, H, d], pos [A, N], f [R / 2]."""
    half = f.numel()
    x = x.double().clone()
    for i in range(half):
        a = pos[0 if axes is None else int(axes[i])].double() * float(f[i])
        c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
        s = -s if inverse else s
        i1, i2 = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        x1, x2 = x[..., i1].clone(), x[..., i2].clone()
        x[..., i1], x[..., i2] = x1 * c - x2 * s, x2 * c + x1 * s
    return x


def turn_bound(x, ref, half, pairs=False):
    """How far a rotated element may be: its rounding, and fp32 arithmetic on the pair: two
    products and a sum (2^-24 each of |x1| + |x2|), sine and cosine of two units in the last
    place (2^-23 of each), the angle within 2^-31 turns (3e-9, below 2^-28)."""
    a = x.double().abs()
    size = a.clone()
    if half:
        i = torch.arange(half)
        i1, i2 = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        size[..., i1] = size[..., i2] = a[..., i1] + a[..., i2]
        rest = torch.ones(x.shape[-1], dtype=torch.bool)
        rest[:2 * half] = False
        size[..., rest] = 0
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 2.0 ** -140
    return U[x.dtype] * ref.abs() * (1 + 2.0 ** -10) + 2.0 ** -21 * size + tiny


def attend(q, k, v, first, scale, causal=True, window=0):
    """Attention of q [t, Hq, d], its first token at position `first`, over k, v [n, Hk, d],
    in 64 bits: outputs, lse and a bound of the outputs' and the lse's errors.

    The bound: scores are fp32 sums of d products, off by g = (d + 4) 2^-24 of the terms'
    magnitudes each, so weights by a factor of e^g at most, and by 2^-22 for the power of two;
    sums of n weights and of n products in fp32 are off by n 2^-24 of their magnitudes.
    With 16-bit inputs weights may be rounded to the inputs' type for the products, and the
    result is rounded once."""
    t, Hq, d = q.shape
    n, Hk = k.shape[0], k.shape[1]
    G, u, dev = Hq // Hk, U[q.dtype], q.device
    q64 = q.double().unflatten(1, (Hk, G))
    x = torch.einsum("thgd,nhd->hgtn", q64, k.double()) * scale
    size = torch.einsum("thgd,nhd->hgtn", q64.abs(), k.double().abs()) * abs(scale)
    at = torch.arange(first, first + t, device=dev)[:, None]
    j = torch.arange(n, device=dev)
    see = torch.ones(t, n, dtype=torch.bool, device=dev)
    if causal:
        see &= j <= at
    if window:
        see &= j > at - window
    x = x.masked_fill(~see, -math.inf)
    some = see.any(1)
    top = x.amax(-1, keepdim=True) if n else torch.zeros(Hk, G, t, 1, device=dev, dtype=torch.float64)
    w = torch.where(see, torch.exp(x - top), 0.0)
    total = w.sum(-1, keepdim=True)
    p = torch.where(some[:, None], w / total, 0.0)
    o = torch.einsum("hgtn,nhd->thgd", p, v.double()).flatten(1, 2)
    mass = torch.einsum("hgtn,nhd->thgd", p, v.double().abs()).flatten(1, 2)
    lse = torch.where(some, (top + torch.log(total)).squeeze(-1), -math.inf).permute(2, 0, 1).flatten(1)
    g = (d + 4) * 2.0 ** -24 * torch.where(see, size, 0.0).amax(-1).permute(2, 0, 1).flatten(1) if n else torch.zeros_like(lse)
    weights = 2 * g + (n + 16) * 2.0 ** -23
    bound = ((u if q.dtype != torch.float32 else 0) + weights[..., None]) * mass + u * o.abs() * (1 + 2 * u) + 2.0 ** -25
    lse_bound = weights + 2.0 ** -22 * lse.abs().nan_to_num(0, 0, 0)
    return o, lse, bound, lse_bound


def near(got, ref, bound, what=""):
    got = got.double()
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    far = (got - ref).abs() - bound
    assert bool((far <= 0).all()), f"{what}: {float(far.max()):.3g} beyond the bound, at {(far == far.max()).nonzero()[0].tolist()}"
