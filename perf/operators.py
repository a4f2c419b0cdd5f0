"""Cases for the operators between a decoder's matrix products: root-mean-square norm with the residual's
addition (and its gradient), counter-based dropout, rotary positions, and the processing of logits.

Each case is run in a plain form (elementary torch operations in 32 bits, rounded once at the end) or,
with `own` set, by the framework's entry points. exact() restates every operator in 64 bits."""

import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EB = {"f32": 4, "bf16": 2, "f16": 2, "s8": 1, "f8": 1}
F8 = torch.float8_e4m3fn
EPS = 1e-6
M32 = 0xFFFFFFFF


# ---- cases -----------------------------------------------------------------------------------------------
def listed():
    return [
        # serving, one request: the norm before a layer's first product for one new token
        dict(name="norm_token", op="norm", rows=1, n=8192, dtype="bf16", out="bf16", residual=True, p=0.0, rstd=False),
        # serving, a batch of new tokens, feeding an 8-bit product
        dict(name="norm_batch_f8", op="norm", rows=256, n=5120, dtype="bf16", out="f8", residual=True, p=0.0,
             rstd=False),
        # a long prompt's (or many prompts') norm
        dict(name="norm_prompt", op="norm", rows=16384, n=8192, dtype="bf16", out="bf16", residual=True, p=0.0,
             rstd=False),
        # training, with dropout on the sub-layer's output before it joins the residual
        dict(name="norm_train", op="norm", rows=8192, n=4096, dtype="bf16", out="bf16", residual=True, p=0.1,
             rstd=True),
        # gradient of a small model's norm, odd row length, 32 bits
        dict(name="norm_grad_odd", op="norm_grad", rows=2049, n=1001, dtype="f32", p=0.0, dsum=True),
        # gradient of the training case's kind, at full size
        dict(name="norm_grad_train", op="norm_grad", rows=16384, n=4096, dtype="bf16", p=0.1, dsum=True),
        # dropout of a small activation of an odd size
        dict(name="dropout_small", op="dropout", rows=37, n=1001, dtype="f32", p=0.5, residual=False),
        # dropout of a large activation, added to the residual
        dict(name="dropout_large", op="dropout", rows=16384, n=8192, dtype="bf16", p=0.1, residual=True),
        # one new token for each of 32 requests: 32 query and 8 key heads, taken from the packed projection
        dict(name="rotary_tokens", op="rotary", batch=32, seq=1, heads=32, kv=8, dim=128, rot=128, dtype="bf16",
             interleaved=False, packed=True, heads_major=False, inverse=False, start=30000, factor=1.0),
        # a long prompt, half of each head rotated in pairs, positions interpolated, written heads first
        dict(name="rotary_prompt", op="rotary", batch=2, seq=16384, heads=32, kv=8, dim=128, rot=64, dtype="bf16",
             interleaved=True, packed=True, heads_major=True, inverse=False, start=0, factor=4.0),
        # one request's logits, with a grammar
        dict(name="logits_one", op="logits", batch=1, vocab=32000, dtype="bf16", history=700, bias=False, mask=True),
        # a batch of requests over a large vocabulary, everything on
        dict(name="logits_batch", op="logits", batch=256, vocab=131072, dtype="bf16", history=4096, bias=True,
             mask=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Most widths are multiples of 64; the rest are odd or ragged."""
    n = _log(rng, lo, hi)
    n = max(64, n // 64 * 64) if rng.random() < 0.6 else n
    return n + 64 if n == 3072 else n


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "dropout", "rotary", "logits"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("norm", "norm_grad"):
        n = _width(rng, 64, 16384)
        rows = max(1, min(_log(rng, 1, 32768), (1 << 26) // n))
        p = rng.choice([0.0, 0.1])
        if op == "norm_grad":
            return dict(op=op, rows=rows, n=n, dtype=dtype, p=p, dsum=rng.random() < 0.7)
        out = rng.choice([dtype, dtype, "f8", "s8"])
        if out == "s8":
            rows = min(rows, 512)
        return dict(op=op, rows=rows, n=n, dtype=dtype, out=out, residual=rng.random() < 0.8, p=p,
                    rstd=rng.random() < 0.5)
    if op == "dropout":
        n = _width(rng, 64, 16384)
        rows = max(1, min(_log(rng, 1, 65536), (1 << 26) // n))
        return dict(op=op, rows=rows, n=n, dtype=dtype, p=rng.choice([0.1, 0.25, 0.5]), residual=rng.random() < 0.5)
    if op == "rotary":
        dim = rng.choice([64, 80, 128, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4, 7])
        seq = rng.choice([1, 1, _log(rng, 2, 16384)])
        batch = max(1, min(_log(rng, 1, 256), (1 << 26) // (seq * (heads + 2 * kv) * dim)))
        return dict(op=op, batch=batch, seq=seq, heads=heads, kv=kv, dim=dim, rot=rng.choice([dim, dim, dim // 2]),
                    dtype=dtype, interleaved=rng.random() < 0.5, packed=rng.random() < 0.5,
                    heads_major=rng.random() < 0.3, inverse=rng.random() < 0.3, start=_log(rng, 1, 500000),
                    factor=rng.choice([1.0, 4.0, 8.0]))
    vocab = _width(rng, 1000, 200000)
    return dict(op=op, batch=max(1, min(_log(rng, 1, 512), (1 << 25) // vocab)), vocab=vocab, dtype=dtype,
                history=_log(rng, 16, 8192), bias=rng.random() < 0.5, mask=rng.random() < 0.7)


# ---- inputs ----------------------------------------------------------------------------------------------
def _turns(case):
    """Turns per position of each pair, in units of 2^-64 turn (whole turns do not matter)."""
    th = [10000.0 ** (-2.0 * i / case["rot"]) / case["factor"] for i in range(case["rot"] // 2)]
    u = [int(t / (2.0 * math.pi) * 2.0 ** 64) % (1 << 64) for t in th]
    return [v - (1 << 64) if v >= 1 << 63 else v for v in u]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = "cuda"
    s = dict(case)
    op = s["op"]
    dt = DT[s["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device=dev).normal_(0.0, std, generator=g)

    def whole(lo, hi, *shape, dtype=torch.int32):
        return torch.empty(*shape, dtype=dtype, device=dev).random_(lo, hi, generator=g)

    s["seed"], s["offset"] = seed * 7919 + 0x1234567890, seed * 31 + 5
    if op == "norm":
        rows, n = s["rows"], s["n"]
        s["x"] = normal(rows, n)
        s["res"] = normal(rows, n, std=2.0) if s["residual"] else None
        s["w"] = normal(n, std=0.1).add_(1.0)
        odt = {"f8": F8, "s8": torch.int8}.get(s["out"]) or DT[s["out"]]
        s["y"] = torch.empty(rows, n, dtype=odt, device=dev)
        s["h"] = torch.empty_like(s["x"]) if s["residual"] or s["p"] else None
        s["scales"] = torch.empty(rows, dtype=torch.float32, device=dev) if s["out"] in ("f8", "s8") else None
        s["rs"] = torch.empty(rows, dtype=torch.float32, device=dev) if s["rstd"] else None
    elif op == "norm_grad":
        rows, n = s["rows"], s["n"]
        s["h"] = normal(rows, n, std=2.0)
        s["dy"] = normal(rows, n, std=0.01)
        s["ds"] = normal(rows, n, std=0.01) if s["dsum"] else None
        s["w"] = normal(n, std=0.1).add_(1.0)
        s["rs"] = (s["h"].float().square().mean(1) + EPS).rsqrt()
        s["dh"] = torch.empty_like(s["h"])
        s["dx"] = torch.empty_like(s["h"]) if s["p"] else None
        s["dw"] = torch.empty(n, dtype=torch.float32, device=dev)
        s["ws"] = None
    elif op == "dropout":
        rows, n = s["rows"], s["n"]
        s["x"] = normal(rows, n)
        s["res"] = normal(rows, n) if s["residual"] else None
        s["y"] = torch.empty_like(s["x"])
    elif op == "rotary":
        b, t, hq, hk, d = s["batch"], s["seq"], s["heads"], s["kv"], s["dim"]
        if s["packed"]:  # queries, keys and values of a token side by side, as one projection writes them
            qkv = normal(b, t, hq + 2 * hk, d)
            s["q"], s["k"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
        else:
            s["q"], s["k"] = normal(b, t, hq, d), normal(b, t, hk, d)
        first = whole(0, s["start"] + 1, b, 1)
        s["pos"] = first + torch.arange(t, dtype=torch.int32, device=dev)
        s["turns"] = torch.tensor(_turns(s), dtype=torch.int64, device=dev)
        s["mscale"] = 1.0 if s["factor"] == 1.0 else 0.1 * math.log(s["factor"]) + 1.0
        if s["heads_major"]:
            s["qo"] = torch.empty(b, hq, t, d, dtype=dt, device=dev).transpose(1, 2)
            s["ko"] = torch.empty(b, hk, t, d, dtype=dt, device=dev).transpose(1, 2)
        else:
            s["qo"], s["ko"] = (torch.empty(b, t, h, d, dtype=dt, device=dev) for h in (hq, hk))
    else:
        b, v, m = s["batch"], s["vocab"], s["history"]
        s["x"] = normal(b, v, std=3.0)
        # tokens of a text repeat: the squares of uniform numbers favour a few of the vocabulary
        u = torch.empty(b, m, device=dev).uniform_(0.0, 1.0, generator=g)
        s["hist"] = (u * u * u * v).to(torch.int32).clamp_(0, v - 1)
        s["lens"] = whole(0, m + 1, b)
        s["prompts"] = (s["lens"].float() * 0.6).to(torch.int32)
        s["rep"] = torch.empty(b, device=dev).uniform_(1.0, 1.5, generator=g)
        s["freq"] = torch.empty(b, device=dev).uniform_(0.0, 0.5, generator=g)
        s["pres"] = torch.empty(b, device=dev).uniform_(0.0, 0.5, generator=g)
        s["bias"] = normal(v, std=0.5, dtype=torch.float32) if s["bias"] else None
        if s["mask"]:
            words = (v + 31) // 32
            s["bits"] = whole(-(1 << 31), 1 << 31, b, words, dtype=torch.int64).to(torch.int32)
            if b > 1:
                s["bits"][whole(0, b, 1).long()] &= 0  # a grammar with no way on
        else:
            s["bits"] = None
        s["y"] = torch.empty_like(s["x"])
        s["token"] = torch.empty(b, dtype=torch.int32, device=dev)
    return s


# ---- the plain forms ---------------------------------------------------------------------------------------
def _product(a, m):
    """High and low 32 bits of a * m for a, m < 2^32 (the int64 product wraps; its bits are right)."""
    p = a * m
    return (p >> 32) & M32, p & M32


def _keep(s, numel):
    """Philox 4x32 with ten rounds (Salmon, Moraes, Dror and Shaw, 2011): element i takes word i % 4 of counter i // 4."""
    c0 = torch.arange((numel + 3) // 4, dtype=torch.int64, device="cuda")
    c0, c1 = c0 & M32, c0 >> 32
    c2 = torch.full_like(c0, s["offset"] & M32)
    c3 = torch.full_like(c0, s["offset"] >> 32)
    k0, k1 = s["seed"] & M32, s["seed"] >> 32
    for _ in range(10):
        h0, l0 = _product(c0, 0xD2511F53)
        h1, l1 = _product(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    words = torch.stack([c0, c1, c2, c3], 1).reshape(-1)[:numel]
    return words >= int(s["p"] * 2.0 ** 32 + 0.5)


def _drop(s, x):
    if not s["p"]:
        return x
    return torch.where(_keep(s, x.numel()).view(x.shape), x * (1.0 / (1.0 - s["p"])), torch.zeros((), device="cuda"))


def _plain_norm(s):
    h = _drop(s, s["x"].float())
    if s["res"] is not None:
        h = h + s["res"].float()
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    y = h * r * s["w"].float()
    got = {"h": h.to(s["x"].dtype) if s["h"] is not None else None, "rstd": r[:, 0] if s["rs"] is not None else None}
    if s["scales"] is None:
        return {**got, "y": y.to(s["y"].dtype)}
    f8 = s["out"] == "f8"
    scale = y.abs().amax(1, keepdim=True) / (448.0 if f8 else 127.0)
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    q = (y / scale).to(F8) if f8 else (torch.round(y / scale) * scale).to(torch.bfloat16)
    return {**got, "y": q, "scales": scale[:, 0]}


def _plain_norm_grad(s):
    h, dy = s["h"].float(), s["dy"].float()
    r = s["rs"][:, None]
    xh = h * r
    g = dy * s["w"].float()
    dh = r * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["ds"] is not None:
        dh = dh + s["ds"].float()
    dx = _drop(s, dh).to(s["h"].dtype) if s["dx"] is not None else None
    return {"dh": dh.to(s["h"].dtype), "dx": dx, "dw": (dy * xh).sum(0)}


def _plain_dropout(s):
    y = _drop(s, s["x"].float())
    if s["res"] is not None:
        y = y + s["res"].float()
    return {"y": y.to(s["x"].dtype)}


def _plain_rotary(s):
    part = (s["pos"].to(torch.int64)[..., None] * s["turns"]) >> 32  # the turn's fraction, in units of 2^-32
    part = ((part + (1 << 31)) & M32) - (1 << 31)
    angle = part.to(torch.float32) * (2.0 * math.pi / 2.0 ** 32)
    c = (torch.cos(angle) * s["mscale"])[:, :, None]
    n = (torch.sin(angle) * (-s["mscale"] if s["inverse"] else s["mscale"]))[:, :, None]

    def turn(x):
        x = x.float()
        rot, rest = x[..., :s["rot"]], x[..., s["rot"]:]
        if s["interleaved"]:
            a, b = rot[..., 0::2], rot[..., 1::2]
            out = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
        else:
            a, b = rot[..., :s["rot"] // 2], rot[..., s["rot"] // 2:]
            out = torch.cat([a * c - b * n, b * c + a * n], -1)
        return torch.cat([out, rest], -1).to(s["q"].dtype)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _allowed(s):
    v = torch.arange(s["vocab"], device="cuda")
    return ((s["bits"][:, v >> 5] >> (v & 31).to(torch.int32)) & 1) != 0


def _plain_logits(s):
    b, v, m = s["batch"], s["vocab"], s["history"]
    x = s["x"].float()
    if s["bias"] is not None:
        x = x + s["bias"]
    at = torch.arange(m, device="cuda")
    given = at < s["lens"][:, None]
    made = given & (at >= s["prompts"][:, None])
    tokens = s["hist"].long()
    seen = torch.zeros(b, v, dtype=torch.int32, device="cuda").scatter_add_(1, tokens, given.to(torch.int32))
    count = torch.zeros(b, v, dtype=torch.int32, device="cuda").scatter_add_(1, tokens, made.to(torch.int32))
    rep = s["rep"][:, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["freq"][:, None] * count.float()
    x = x - s["pres"][:, None] * (count > 0).float()
    if s["bits"] is not None:
        x = torch.where(_allowed(s), x, torch.full((), -math.inf, device="cuda"))
    top = x.amax(1, keepdim=True)
    token = torch.where(x == top, torch.arange(v, device="cuda"), v).amin(1)
    token = torch.where(top[:, 0] == -math.inf, -1, token)
    return {"y": x.to(s["x"].dtype), "token": token.to(torch.int32)}


# ---- the framework's entry points --------------------------------------------------------------------------
def _own_run(s):
    import transpose_heroes_gb300 as hf

    op = s["op"]
    if op == "norm":
        drop = hf.Dropout(s["p"], s["seed"], s["offset"]) if s["p"] else None
        hf.rms_norm(s["x"], s["y"], weight=s["w"], residual=s["res"], sum_out=s["h"], rstd=s["rs"], eps=EPS, dropout=drop,
                    scales=s["scales"])
        y = s["y"] if s["out"] != "s8" else (s["y"].float() * s["scales"][:, None]).to(torch.bfloat16)
        got = {"h": s["h"], "rstd": s["rs"], "y": y}
        return got if s["scales"] is None else {**got, "scales": s["scales"]}
    if op == "norm_grad":
        drop = hf.Dropout(s["p"], s["seed"], s["offset"]) if s["p"] else None
        if s["ws"] is None:  # the scratch of a training program, allocated once
            s["ws"] = torch.empty(hf.rms_norm_workspace_size(s["rows"], s["n"]), dtype=torch.uint8, device="cuda")
        hf.rms_norm_backward(s["dy"], s["h"], s["rs"], s["dh"], weight=s["w"], dsum=s["ds"], dx=s["dx"], dropout=drop,
                             dweight=s["dw"], workspace=s["ws"])
        return {"dh": s["dh"], "dx": s["dx"], "dw": s["dw"]}
    if op == "dropout":
        hf.dropout(s["x"], s["y"], hf.Dropout(s["p"], s["seed"], s["offset"]), residual=s["res"])
        return {"y": s["y"]}
    if op == "rotary":
        hf.rotary(s["q"], s["qo"], s["pos"], s["turns"], k=s["k"], k_out=s["ko"], interleaved=s["interleaved"],
                  scale=s["mscale"], inverse=s["inverse"])
        return {"q": s["qo"], "k": s["ko"]}
    hf.logits_process(s["x"], s["y"], bias=s["bias"], history=s["hist"], lengths=s["lens"], prompt_lengths=s["prompts"],
                      repetition=s["rep"], frequency=s["freq"], presence=s["pres"], mask=s["bits"], token=s["token"])
    return {"y": s["y"], "token": s["token"]}


def run(s):
    if own:
        return _own_run(s)
    return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "dropout": _plain_dropout, "rotary": _plain_rotary,
            "logits": _plain_logits}[s["op"]](s)


# ---- what a pass cannot do without ---------------------------------------------------------------------------
def work(case):
    op, e = case["op"], EB[case["dtype"]]
    if op == "norm":
        el = case["rows"] * case["n"]
        summed = case["residual"] or case["p"]
        per = e + (e if case["residual"] else 0) + (e if summed else 0) + EB[case["out"]]
        side = case["n"] * e + case["rows"] * 4 * ((case["out"] in ("f8", "s8")) + case["rstd"])
        return {"bytes": el * per + side, "flops": el * (5 + (1 if case["residual"] else 0))}
    if op == "norm_grad":
        el = case["rows"] * case["n"]
        per = e * (3 + case["dsum"] + (case["p"] > 0))
        return {"bytes": el * per + case["n"] * (e + 4) + case["rows"] * 4, "flops": el * 10}
    if op == "dropout":
        el = case["rows"] * case["n"]
        return {"bytes": el * e * (2 + case["residual"]), "flops": el * (1 + case["residual"])}
    if op == "rotary":
        tokens = case["batch"] * case["seq"]
        el = tokens * (case["heads"] + case["kv"]) * case["dim"]
        return {"bytes": 2 * el * e + tokens * 4 + case["rot"] * 4,
                "flops": tokens * (case["heads"] + case["kv"]) * case["rot"] * 3}
    b, v = case["batch"], case["vocab"]
    side = b * case["history"] * 4 * 0.5 + (v * 4 if case["bias"] else 0) + (b * ((v + 31) // 32) * 4 if case["mask"] else 0)
    return {"bytes": 2 * b * v * e + side + b * 24, "flops": b * v * 2}


# ---- the operators in 64 bits ----------------------------------------------------------------------------------
def _kept_exactly(s, numel):
    """The same generator, with its 32 x 32 bit products put together from 16-bit halves."""
    i = torch.arange(numel, dtype=torch.int64, device="cuda")
    q = i.div(4, rounding_mode="floor")
    q = q[::4].contiguous()
    x = [q % 2 ** 32, q // 2 ** 32, torch.full_like(q, s["offset"] % 2 ** 32), torch.full_like(q, s["offset"] // 2 ** 32)]

    def wide(a, m):
        a0, a1, m0, m1 = a % 65536, a // 65536, m % 65536, m // 65536
        mid = a0 * m1 + (a0 * m0) // 65536
        mid2 = a1 * m0 + mid % 65536
        return a1 * m1 + mid // 65536 + mid2 // 65536, (mid2 % 65536) * 65536 + (a0 * m0) % 65536

    for r in range(10):
        key = [(s["seed"] % 2 ** 32 + r * 0x9E3779B9) % 2 ** 32, (s["seed"] // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32]
        (h0, l0), (h1, l1) = wide(x[0], 0xD2511F53), wide(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ key[0], l1, h0 ^ x[3] ^ key[1], l0]
    word = torch.empty(4 * q.numel(), dtype=torch.int64, device="cuda")
    for k in range(4):
        word[k::4] = x[k]
    return word[:numel] >= round(s["p"] * 2 ** 32)


def _dropped(s, x):
    if not s["p"]:
        return x
    kept = _kept_exactly(s, x.numel()).reshape(x.shape)
    return (x / (1.0 - s["p"])).masked_fill_(~kept, 0.0)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "norm":
        h = _dropped(s, s["x"].double())
        if s["res"] is not None:
            h += s["res"]
        r = 1.0 / (h.pow(2).sum(1) / s["n"] + EPS).sqrt()
        y = h * s["w"].double() * r[:, None]
        got = {"h": h if s["h"] is not None else None, "rstd": r if s["rs"] is not None else None, "y": y}
        if s["scales"] is None:
            return got
        scale = y.abs().max(1).values / (448.0 if s["out"] == "f8" else 127.0)
        return {**got, "y": y / scale[:, None] if s["out"] == "f8" else y, "scales": scale}
    if op == "norm_grad":
        r = s["rs"].double()[:, None]
        xh, dy = s["h"].double() * r, s["dy"].double()
        g = dy * s["w"].double()
        dh = r * g - r * xh * ((g * xh).sum(1, keepdim=True) / s["n"])
        if s["ds"] is not None:
            dh += s["ds"]
        return {"dh": dh, "dx": _dropped(s, dh) if s["dx"] is not None else None, "dw": (dy * xh).sum(0)}
    if op == "dropout":
        y = _dropped(s, s["x"].double())
        return {"y": y if s["res"] is None else y + s["res"].double()}
    if op == "rotary":
        pair = torch.arange(s["rot"] // 2, dtype=torch.float64, device="cuda")
        angle = s["pos"].double()[..., None] * (10000.0 ** (-2.0 * pair / s["rot"]) / s["factor"])
        z = torch.polar(torch.full_like(angle, s["mscale"]), -angle if s["inverse"] else angle)[:, :, None]

        def turn(x):
            out = x.double()
            h = s["rot"] // 2
            a, b = (slice(0, s["rot"], 2), slice(1, s["rot"], 2)) if s["interleaved"] else (slice(0, h), slice(h, s["rot"]))
            w = torch.complex(out[..., a], out[..., b]) * z
            out = out.clone()
            out[..., a], out[..., b] = w.real, w.imag
            return out

        return {"q": turn(s["q"]), "k": turn(s["k"])}
    x = s["x"].double()
    if s["bias"] is not None:
        x = x + s["bias"].double()
    row = torch.arange(s["batch"], device="cuda")[:, None].expand(-1, s["history"])
    place = torch.arange(s["history"], device="cuda").expand(s["batch"], -1)
    inside = place < s["lens"][:, None]
    late = inside & (place >= s["prompts"][:, None])
    key = row * s["vocab"] + s["hist"].long()
    total = s["batch"] * s["vocab"]
    seen = torch.bincount(key[inside], minlength=total).view(x.shape) > 0
    count = torch.bincount(key[late], minlength=total).view(x.shape).double()
    rep = s["rep"].double()[:, None].expand_as(x)
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["freq"].double()[:, None] * count - s["pres"].double()[:, None] * count.clamp(max=1.0)
    if s["bits"] is not None:
        shifts = torch.arange(32, device="cuda")
        open_ = ((s["bits"].long()[:, :, None] >> shifts) & 1).flatten(1)[:, :s["vocab"]].bool()
        x = x.masked_fill(~open_, -math.inf)
    return {"y": x, "token": None}
