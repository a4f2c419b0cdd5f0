"""Plain 64-bit statements of the paged cache's operators, for the tests, and the inputs that the tests give them.

Error bounds use the unit roundoffs of layer_reference and hold for any order of summation."""

import math

import numpy as np
import torch

from layer_reference import HALF_ULP, TINY, U

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "f8": torch.float8_e4m3fn}
F8_MAX = 448.0


class Cache:
    """A cache whose pages lie in a random order. Everything that is no entry of a sequence is NaN, and stays so: a kernel that
    reads it shows it."""

    def __init__(self, rng, lengths, new, kv, dim, page, dtype, device, heads_major=False, spare=3, layers=None, order="random",
                 k_scale=1.0, v_scale=1.0, pad=0):
        self.lengths, self.new, self.kv, self.dim, self.page = list(lengths), new, kv, dim, page
        self.dtype, self.k_scale, self.v_scale = dtype, k_scale, v_scale
        b = len(self.lengths)
        width = max(1, max(-(-(n + new) // page) for n in self.lengths))
        total = b * width + spare
        ids = rng.permutation(total) if order == "random" else np.arange(total)
        self.table = torch.from_numpy(ids[:b * width].reshape(b, width).astype(np.int32)).to(device)
        self.width, self.total = width, total
        lead = () if layers is None else (layers,)
        shape = (total, kv, page, dim + pad) if heads_major else (total, page, kv, dim + pad)
        self.stores = [torch.full((*lead, *shape), math.nan, dtype=torch.float32).to(DT[dtype]).to(device) for _ in range(2)]
        views = [s[..., :dim] for s in self.stores]
        self.k, self.v = [s.transpose(-3, -2) if heads_major else s for s in views]
        self.len = torch.tensor(self.lengths, dtype=torch.int32, device=device)

    def raw(self, t):
        return t.view(torch.uint8) if self.dtype == "f8" else t

    def where(self, b, entries):
        e = torch.as_tensor(entries, dtype=torch.int64, device=self.table.device)
        return self.table[b].long()[e // self.page], e % self.page

    def put(self, b, entries, k, v):
        """k, v [n, kv, dim] (any float type) as entries of sequence b."""
        page, place = self.where(b, entries)
        for store, x in ((self.k, k), (self.v, v)):
            self.raw(store)[..., page, place, :, :] = self.raw(x.to(DT[self.dtype]).to(store.device))

    def get(self, b, entries):
        """float64 [n, kv, dim] of keys and values, on the CPU."""
        page, place = self.where(b, entries)
        return [(self.raw(t)[page, place].view(t.dtype).double() * s).cpu()
                for t, s in ((self.k, self.k_scale), (self.v, self.v_scale))]


def normal(rng, shape, dtype, std=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * std).to(DT[dtype])


def filled(rng, lengths, counts, new, kv, dim, page, dtype, device, std=1.0, **kw):
    """A cache that holds random entries for every sequence's length and its new tokens."""
    c = Cache(rng, lengths, new, kv, dim, page, dtype, device, **kw)
    for b, n in enumerate(lengths):
        m = n + counts[b]
        if m:
            k, v = (normal(rng, (m, kv, dim), "f32", std / s) for s in (c.k_scale, c.v_scale))
            c.put(b, range(m), k, v)
    return c


def random_tree(rng, n):
    """Parents of n nodes; the first is the root."""
    return [-1] + [int(rng.integers(0, c)) for c in range(1, n)]


def sees_of(parents):
    """[n, n] truth values: whether a node sees another."""
    n = len(parents)
    s = np.zeros((n, n), bool)
    for c in range(n):
        u = c
        while u >= 0:
            s[c, u] = True
            u = parents[u]
    return s


def packed(sees):
    """[..., n, m] truth values as words of 32 bits."""
    n = sees.shape[-1]
    words = (n + 31) // 32
    bits = np.zeros((*sees.shape[:-1], words * 32), np.uint64)
    bits[..., :n] = sees
    w = (bits.reshape(*sees.shape[:-1], words, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return torch.from_numpy(w.astype(np.uint32).view(np.int32))


def attention(q, k, v, sees, scale):
    """q [t, heads, dim], k and v [n, kv, dim] in float64, sees [t, n] -> out, lse and the bound of the errors of an f32 kernel
    that rounds weights to `weights` bits, before out's own rounding: a function of the half step of the weights' type."""
    t, heads, dim = q.shape
    kv = k.shape[1]
    seen = torch.as_tensor(sees)
    qg = q.view(t, kv, heads // kv, dim).permute(1, 2, 0, 3)  # [kv, group, t, dim]
    kk, vv = k.permute(1, 2, 0)[:, None], v.permute(1, 0, 2)[:, None]
    clean = lambda x: torch.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0)  # noqa: E731
    s = (qg @ clean(kk)) * scale
    size = (qg.abs() @ clean(kk).abs()) * scale  # sums of |terms|
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(s - top)
    total = e.sum(-1, keepdim=True)
    p = torch.where(total > 0, e / total, torch.zeros_like(e))
    out = (p @ clean(vv)).permute(2, 0, 1, 3).reshape(t, heads, dim)
    lse = (top + torch.log(total))[..., 0].permute(2, 0, 1).reshape(t, heads)
    n = k.shape[0]
    # a score: products and their sum in any order, the scale and the change of base, and the subtraction of the maximum
    es = ((dim + 6) * U * size.masked_fill(~seen, 0.0).amax(-1, keepdim=True) + 4 * U * top.abs())
    spread = (p @ clean(vv).abs())
    # weights: the scores' errors and the exponential's 2^-21; both sums over the entries; a few factors of the join
    e32 = ((2 * es + 2.0 ** -20 + (2 * n + 64) * U) * spread).permute(2, 0, 1, 3).reshape(t, heads, dim)
    widest = clean(vv).abs().sum(-2, keepdim=True).expand_as(spread)
    each = spread.permute(2, 0, 1, 3).reshape(t, heads, dim)
    widest = widest.permute(2, 0, 1, 3).reshape(t, heads, dim)
    elen = (es + 2.0 ** -20 + (n + 64) * U)[..., 0].permute(2, 0, 1).reshape(t, heads) + 4 * U * lse.abs().nan_to_num(posinf=0.0)

    def bound(weights):
        if weights is None:
            return e32
        # each weight is off by half a step, or by half of the smallest step where it is below the type's normal numbers
        # (the largest weight of a row is at least 1 in the kernel's units, so its sum is too)
        return e32 + HALF_ULP[weights] * (1 + 2.0 ** -8) * each + TINY[weights] * widest

    return out, lse, bound, elen


def turned(x, positions, turns, interleaved=False, scale=1.0):
    """x [t, heads, dim] float64 by positions [t] * turns (int64 words): exact angles, and the bound of an f32 kernel's error."""
    pairs = len(turns)
    frac = [[((int(p) * int(u)) % (1 << 64)) / 2.0 ** 64 for u in turns] for p in positions]
    a = 2 * math.pi * torch.tensor(frac, dtype=torch.float64).view(len(positions), 1, pairs)
    c, s = torch.cos(a) * scale, torch.sin(a) * scale
    i = torch.arange(pairs)
    u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
    out, err = x.clone(), torch.zeros_like(x)
    out[..., u] = x[..., u] * c - x[..., v] * s
    out[..., v] = x[..., v] * c + x[..., u] * s
    # the angle is held to 2^-32 turn, its cosine to 4 ulp, the products and their sum to 3 roundings
    e = (8 * U + 2 * math.pi * 2.0 ** -31) * abs(scale) * (x[..., u].abs() + x[..., v].abs())
    err[..., u], err[..., v] = e, e
    return out, err


def rounding(x, dtype):
    """Half a step of the type at each value."""
    if dtype == "f8":
        return torch.clamp(x.abs() * 2.0 ** -4, min=2.0 ** -10)
    return x.abs() * HALF_ULP[dtype] + TINY[dtype]


def accept(tokens, parents, picks, count):
    path = []
    if count:
        path = [0]
        while True:
            c = path[-1]
            follow = [d for d in range(c + 1, count) if parents[d] == c and picks[c] >= 0 and tokens[d] == picks[c]]
            if not follow:
                break
            path.append(follow[0])
    return path
