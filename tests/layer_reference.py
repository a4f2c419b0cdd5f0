"""Plain 64-bit statements of the fusions between a decoder's matrix products, in numpy, for the tests.

Inputs are numpy float64 arrays that hold the operands' (already rounded) values. Error bounds use the
unit roundoff U = 2^-24 of f32 and hold for any order of summation: a sum of k terms t is within
k U sum|t| of its value."""

import math

import numpy as np

U = 2.0 ** -24
# half a unit in the last of p significant bits, relative to the value: 2^-p
HALF_ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
# the spacing of the smallest values of a type, halved
TINY = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}


def philox(seed, offset, quad):
    """Philox4x32-10 words [len(quad), 4] for the counters `quad` (Salmon et al., SC 2011), with Python's
    64-bit products."""
    q = np.asarray(quad, dtype=np.uint64)
    m32 = np.uint64(0xFFFFFFFF)
    s32 = np.uint64(32)
    c = [q & m32, q >> s32, np.full_like(q, offset & 0xFFFFFFFF), np.full_like(q, (offset >> 32) & 0xFFFFFFFF)]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> s32) ^ c[1] ^ np.uint64(k[0]), p1 & m32, (p0 >> s32) ^ c[3] ^ np.uint64(k[1]), p0 & m32]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, -1)


def keep(p, seed, offset, numel):
    words = philox(seed, offset, np.arange((numel + 3) // 4)).reshape(-1)[:numel]
    return words >= np.uint64(int(math.floor(p * 2.0 ** 32 + 0.5)))


def drop_scale(p):
    """f32(1 / (1 - p)): the factor is an f32 by definition."""
    return float(np.float32(1.0 / (1.0 - p))) if p < 1 else 0.0


def drop(x, d):
    if d is None:
        return x
    p, seed, offset = d
    k = keep(p, seed, offset, x.size).reshape(x.shape)
    return np.where(k, np.where(k, x, 0.0) * drop_scale(p), 0.0)


def rms_norm(x, w, residual=None, w_offset=0.0, eps=1e-6, d=None):
    """(h, r, y) and the bound of |h - f32 h| per element, |r| relative, |y| per element (f32, before output
    rounding)."""
    n = x.shape[-1]
    dx = drop(x, d)
    h = dx if residual is None else residual + dx
    eh = 2 * U * (np.abs(dx) + (0 if residual is None else np.abs(residual)))
    r = 1.0 / np.sqrt((h * h).mean(-1) + eps)
    # relative error of mean(h^2): the sum's order, each square, the division and eps; and that of h's own error
    er = 0.5 * ((n + 4) * U + 2 * (np.abs(h) * eh).sum(-1) / np.maximum((h * h).sum(-1), 1e-300)) + 4 * U
    ww = w + w_offset
    y = h * r[..., None] * ww
    ey = np.abs(y) * (er[..., None] + 4 * U) + eh * r[..., None] * np.abs(ww)
    return h, r, y, eh, er, ey


def rms_norm_backward(dy, h, rstd, w, w_offset=0.0, dsum=None, d=None):
    n = h.shape[-1]
    ww = w + w_offset
    g, xh = dy * ww, h * rstd[..., None]
    mean, mag = (g * xh).mean(-1, keepdims=True), np.abs(g * xh).mean(-1, keepdims=True)
    dh = rstd[..., None] * (g - xh * mean)
    edh = rstd[..., None] * (8 * U * np.abs(g) + np.abs(xh) * mag * (n + 12) * U)
    if dsum is not None:
        dh = dh + dsum
        edh = edh + 2 * U * (np.abs(dsum) + np.abs(dh))
    dx = drop(dh, d)
    edx = np.where(dx != 0, (edh + 2 * U * np.abs(dh)) * (1 if d is None else drop_scale(d[0])), 0.0)
    t = (dy * xh).reshape(-1, n)
    dw, edw = t.sum(0), (t.shape[0] + 8) * U * np.abs(t).sum(0)
    return dh, dx, dw, edh, edx, edw


def turns_of(rot, base=10000.0, factor=1.0):
    th = [base ** (-2.0 * i / rot) / factor for i in range(rot // 2)]
    return np.array([int(t / (2 * math.pi) * 2.0 ** 64) for t in th], dtype=np.uint64)


def rotary(x, positions, turns, interleaved=False, scale=1.0, inverse=False):
    """x [batch, seq, heads, dim], positions [batch, seq]; also the bound of the f32 result's error."""
    half = len(turns)
    with np.errstate(over="ignore"):
        frac = positions.astype(np.int64).astype(np.uint64)[..., None] * turns  # mod 2^64
    angle = frac.astype(np.float64) / 2.0 ** 64 * 2 * math.pi
    c, s = np.cos(angle)[:, :, None] * scale, np.sin(angle)[:, :, None] * scale * (-1 if inverse else 1)
    out = x.copy()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    out[..., a], out[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    # the angle: 2^-32 turn cut off and an f32 rounding of at most half a turn (pi U); cos and sin: 2 ulp
    # (4 U); scale, products and sum: 4 roundings
    e = np.zeros_like(x)
    k = (2 * math.pi * 2.0 ** -32 + math.pi * U + 4 * U + 4 * U) * abs(scale)
    e[..., a] = e[..., b] = k * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return out, e


def logits(x, bias=None, history=None, lengths=None, prompts=None, repetition=None, frequency=None, presence=None,
           allowed=None):
    """x: float32 values. The steps in f32, each a single IEEE operation, so that the result is exact; and the
    greedy token."""
    f = np.float32
    l = x.astype(f)
    if bias is not None:
        l = l + np.broadcast_to(bias, l.shape).astype(f)
    b, v = l.shape
    for i in range(b):
        if history is None:
            continue
        m = history.shape[1]
        n = m if lengths is None else int(min(max(lengths[i], 0), m))
        pl = 0 if prompts is None else int(prompts[i])
        seen, count = np.zeros(v, bool), np.zeros(v, np.int64)
        for j in range(n):
            t = int(history[i, j])
            if 0 <= t < v:
                seen[t] = True
                count[t] += j >= pl
        rep = f(1) if repetition is None else f(repetition[i])
        fr, pr = (f(0) if q is None else f(q[i]) for q in (frequency, presence))
        with np.errstate(invalid="ignore", over="ignore"):
            l[i] = np.where(seen, np.where(l[i] > 0, l[i] / rep, l[i] * rep), l[i])
            l[i] = np.where(seen, l[i] - fr * count.astype(f), l[i])
            l[i] = np.where(count > 0, l[i] - pr, l[i])
    if allowed is not None:
        l = np.where(np.broadcast_to(allowed, l.shape), l, f(-np.inf))
    token = np.full(b, -1, np.int32)
    for i in range(b):
        ok = l[i] > -np.inf  # false for NaN
        if ok.any():
            top = l[i][ok].max()
            token[i] = int(np.flatnonzero(ok & (l[i] == top))[0])
    return l, token
