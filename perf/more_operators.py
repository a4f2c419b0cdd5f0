"""Cases for a decoder's paged cache: appending keys and values with the position rotation on the way, attention of
new tokens (single ones, a prompt, or a tree of drafted ones) over the cache, and the acceptance of a drafted
branch, which moves its entries together.

Each case is run in a plain form (elementary torch operations in 32 bits, rounded once at the end) or,
with `own` set, by the framework's entry points. exact() restates the computed outputs in 64 bits.

A cache is [pages, page, kv, dim] (with layers before it for the acceptance); entry i of sequence b lies in page
pages[b, i // page] at place i % page. A tree's node 0 is the last known token; parents come before their children."""

import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "f8": torch.float8_e4m3fn}
EB = {"f32": 4, "bf16": 2, "f16": 2, "f8": 1}
F8_MAX = 448.0
K_SCALE, V_SCALE = 0.02, 0.015
VOCAB = 32000
M32 = 0xFFFFFFFF


# ---- cases -----------------------------------------------------------------------------------------------
def listed():
    return [
        # one new token for each of 32 requests, before a layer's attention
        dict(name="append_tokens", op="append", batch=32, seq=1, heads=32, kv=8, dim=128, rot=128, dtype="bf16", cache="bf16",
             page=16, length=4096, interleaved=False, tree=False, heads_major=False),
        # drafted trees of 24 nodes for 16 requests, at positions by depth, into an 8-bit cache; half of each head turns
        dict(name="append_trees_f8", op="append", batch=16, seq=24, heads=32, kv=8, dim=128, rot=64, dtype="bf16", cache="f8",
             page=32, length=2048, interleaved=True, tree=True, heads_major=True),
        # two long prompts, written whole
        dict(name="append_prompt", op="append", batch=2, seq=8192, heads=32, kv=8, dim=128, rot=128, dtype="bf16", cache="bf16",
             page=64, length=0, interleaved=False, tree=False, heads_major=False),
        # one request's next token
        dict(name="attend_token", op="attend", batch=1, seq=1, heads=32, kv=8, dim=128, dtype="bf16", cache="bf16", page=16,
             length=4096, tree=False, lse=False, heads_major=False),
        # a batch of requests of unequal lengths, one new token each
        dict(name="attend_batch", op="attend", batch=64, seq=1, heads=32, kv=8, dim=128, dtype="bf16", cache="bf16", page=16,
             length=8192, tree=False, lse=False, heads_major=False),
        # small drafted trees over an 8-bit cache
        dict(name="attend_trees_f8", op="attend", batch=32, seq=8, heads=32, kv=8, dim=128, dtype="bf16", cache="f8", page=32,
             length=16384, tree=True, lse=False, heads_major=True),
        # larger drafted trees
        dict(name="attend_trees", op="attend", batch=16, seq=48, heads=32, kv=8, dim=128, dtype="bf16", cache="bf16", page=64,
             length=16384, tree=True, lse=False, heads_major=False),
        # 32 bits, with heads and pages of odd sizes and the softmax's statistics, as a small model's check has them
        dict(name="attend_odd", op="attend", batch=3, seq=5, heads=6, kv=2, dim=40, dtype="f32", cache="f32", page=7,
             length=1001, tree=True, lse=True, heads_major=False),
        # prompts over an empty cache: every token sees those before it
        dict(name="attend_prompt", op="attend", batch=4, seq=4096, heads=32, kv=8, dim=128, dtype="bf16", cache="bf16", page=64,
             length=0, tree=False, lse=False, heads_major=False),
        # one request's draft of 16 nodes, in a model of 16 layers
        dict(name="accept_one", op="accept", batch=1, seq=16, layers=16, kv=8, dim=128, cache="bf16", page=16, length=256,
             kept=4, heads_major=False),
        # a batch of larger drafts, entries of odd sizes
        dict(name="accept_odd", op="accept", batch=9, seq=33, layers=3, kv=3, dim=50, cache="f16", page=5, length=100, kept=6,
             heads_major=True),
        # a batch of larger drafts
        dict(name="accept_batch", op="accept", batch=64, seq=48, layers=16, kv=8, dim=128, cache="bf16", page=64, length=200,
             kept=8, heads_major=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "accept"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    cache = rng.choice([dtype, dtype, "f8"])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 4, 4, 7, 8])
    dim = rng.choice([64, 80, 128, 128, 128, 256])
    page = rng.choice([16, 16, 32, 64, 128, 24, _log(rng, 1, 200)])
    major = rng.random() < 0.4
    if op == "append":
        seq = rng.choice([1, 1, _log(rng, 2, 64), _log(rng, 64, 8192)])
        batch = max(1, min(_log(rng, 1, 256), (1 << 24) // (seq * kv * dim)))
        return dict(op=op, batch=batch, seq=seq, heads=heads, kv=kv, dim=dim, rot=rng.choice([dim, dim, dim // 2]), dtype=dtype,
                    cache=cache, page=page, length=min(_log(rng, 1, 8192), (1 << 27) // (batch * kv * dim)), interleaved=rng.random() < 0.5,
                    tree=seq <= 64 and rng.random() < 0.5, heads_major=major)
    if op == "attend":
        seq = rng.choice([1, 1, _log(rng, 2, 64), _log(rng, 2, 64), _log(rng, 64, 4096)])
        if dtype == "f32":
            seq = min(seq, 64)
        batch = max(1, min(_log(rng, 1, 128), (1 << 23) // (seq * heads * dim)))
        most = min((1 << 29) // (batch * kv * dim), (1 << 30) // (batch * heads * seq) - seq, 65536)
        length = _log(rng, 1, max(2, most)) if rng.random() < 0.9 else 0
        return dict(op=op, batch=batch, seq=seq, heads=heads, kv=kv, dim=dim, dtype=dtype, cache=cache, page=page,
                    length=max(0, min(length, most)), tree=seq <= 256 and rng.random() < 0.6, lse=rng.random() < 0.4, heads_major=major)
    seq, layers = _log(rng, 4, 256), _log(rng, 1, 16)
    batch = max(1, min(_log(rng, 1, 128), (1 << 27) // (layers * kv * dim * (seq + 256))))
    return dict(op=op, batch=batch, seq=seq, layers=layers, kv=kv, dim=dim, cache=cache, page=page, length=_log(rng, 1, 256),
                kept=rng.randint(1, max(1, min(12, seq // 4))), heads_major=major)


def _spread(lo, hi, n):
    """n whole numbers over lo..hi, the greatest among them."""
    return [hi - (hi - lo) * i // n for i in range(n)]


def _lengths(case):
    return _spread(case["length"] // 4, case["length"], case["batch"])


def _counts(case):
    """New tokens of each sequence: some of the batch have fewer than the others."""
    few = case["seq"] if case["seq"] > 64 else (case["seq"] + 1) // 2
    return _spread(few, case["seq"], case["batch"])


def _kept(case):
    """Entries of each accepted branch, node 0 among them."""
    return _spread(1, case["kept"], case["batch"])


# ---- inputs ----------------------------------------------------------------------------------------------
def _turns(rot):
    """Turns per position of each pair, in units of 2^-64 turn (whole turns do not matter)."""
    u = [int(10000.0 ** (-2.0 * i / rot) / (2.0 * math.pi) * 2.0 ** 64) % (1 << 64) for i in range(rot // 2)]
    return [v - (1 << 64) if v >= 1 << 63 else v for v in u]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = "cuda"
    s = dict(case)
    op, b, n = s["op"], s["batch"], s["seq"]

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device=dev).normal_(0.0, std, generator=g)

    def whole(lo, hi, *shape):
        return torch.empty(*shape, dtype=torch.int32, device=dev).random_(lo, hi, generator=g)

    def mixed(values):
        order = torch.randperm(b, device=dev, generator=g)
        return torch.tensor(values, dtype=torch.int32, device=dev)[order]

    s["lengths"], s["counts"] = mixed(_lengths(s)), mixed(_counts(s))
    width = (s["length"] + n + s["page"] - 1) // s["page"]
    s["pages"] = torch.randperm(b * width, device=dev, generator=g).to(torch.int32).view(b, width)
    lead = (s["layers"],) if op == "accept" else ()
    for name, scale in (("k_cache", K_SCALE), ("v_cache", V_SCALE)):
        shape = (b * width, s["kv"], s["page"], s["dim"]) if s["heads_major"] else (b * width, s["page"], s["kv"], s["dim"])
        if s["cache"] == "f8":
            c = torch.empty(*lead, *shape, dtype=DT["f8"], device=dev)
            for part in (c if lead else [c]):
                part.copy_(normal(*shape, std=1.0 / scale, dtype=torch.bfloat16).clamp_(-F8_MAX, F8_MAX))
        else:
            c = normal(*lead, *shape, dtype=DT[s["cache"]])
        s[name] = c.transpose(-3, -2) if s["heads_major"] else c

    # every node's parent lies before it; the accepted branch of the largest kept is chain[0] = 0, chain[1], ...
    parents = (torch.rand(b, n, device=dev, generator=g) * torch.arange(n, device=dev)).to(torch.int32)
    parents[:, 0] = -1
    if op == "accept":
        kept = mixed(_kept(s))
        s["counts"] = torch.full((b,), n, dtype=torch.int32, device=dev)
        # its nodes lie behind the places that they move to
        chain = [0] + [s["kept"] + (n - s["kept"]) * i // s["kept"] for i in range(s["kept"] - 1)]
        for i in range(1, len(chain)):
            parents[:, chain[i]] = chain[i - 1]
        s["tokens"], s["picks"] = whole(0, VOCAB, b, n), whole(0, VOCAB, b, n)
        for i in range(1, len(chain)):
            s["picks"][:, chain[i - 1]] = torch.where(i < kept, s["tokens"][:, chain[i]], s["picks"][:, chain[i - 1]])
        s["path"] = torch.empty(b, n, dtype=torch.int32, device=dev)
        s["accepted"], s["next"] = (torch.empty(b, dtype=torch.int32, device=dev) for _ in range(2))
    s["parents"] = parents
    if op == "accept" or s["tree"]:  # which nodes lie between a node and the root, and their number
        above = torch.eye(n, dtype=torch.bool, device=dev).expand(b, n, n).clone()
        for i in range(1, n):
            above[:, i] |= above.gather(1, parents[:, i].long()[:, None, None].expand(b, 1, n))[:, 0]
        s["above"] = above
        words = (n + 31) // 32
        bits = torch.zeros(b, n, words * 32, dtype=torch.int64, device=dev)
        bits[:, :, :n] = above
        bits = (bits.view(b, n, words, 32) << torch.arange(32, device=dev)).sum(-1)
        s["mask"] = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)
        depth = above.sum(-1, dtype=torch.int32) - 1
    else:
        s["mask"] = None
        depth = torch.arange(n, dtype=torch.int32, device=dev).expand(b, n)
    if op == "accept":
        return s
    dt, h, kv, d = DT[s["dtype"]], s["heads"], s["kv"], s["dim"]
    qkv = normal(b, n, h + 2 * kv, d, dtype=dt)  # queries, keys and values of a token side by side, as one projection writes them
    s["q"], s["k"], s["v"] = qkv[:, :, :h], qkv[:, :, h:h + kv], qkv[:, :, h + kv:]
    s["out"] = torch.zeros(b, n, h, d, dtype=dt, device=dev)
    if op == "append":
        s["turns"] = torch.tensor(_turns(s["rot"]), dtype=torch.int64, device=dev)
        s["positions"] = s["lengths"][:, None] + depth if s["tree"] else None
    else:
        s["q"].mul_(2.0)
        s["stats"] = torch.zeros(b, n, h, dtype=torch.float32, device=dev) if s["lse"] else None
        s["ws"] = None
    return s


# ---- the plain forms ---------------------------------------------------------------------------------------
def _place(s, slot):
    """Page and place of slots [batch, n] of the cache."""
    slot = slot.long()
    return torch.gather(s["pages"], 1, slot // s["page"]).long(), slot % s["page"]


def _bits(c):
    return c.view(torch.uint8) if c.dtype == DT["f8"] else c


def _coded(s, x, scale):
    """x as the cache holds it."""
    if s["cache"] == "f8":
        return (x / scale).clamp(-F8_MAX, F8_MAX).to(DT["f8"])
    return x.to(DT[s["cache"]])


def _positions(s):
    if s["positions"] is not None:
        return s["positions"]
    return s["lengths"][:, None] + torch.arange(s["seq"], dtype=torch.int32, device="cuda")


def _plain_append(s):
    part = (_positions(s).to(torch.int64)[..., None] * s["turns"]) >> 32  # the turn's fraction, in units of 2^-32
    part = ((part + (1 << 31)) & M32) - (1 << 31)
    angle = part.to(torch.float32) * (2.0 * math.pi / 2.0 ** 32)
    c, n = torch.cos(angle)[:, :, None], torch.sin(angle)[:, :, None]

    def turn(x):
        x = x.float()
        rot, rest = x[..., :s["rot"]], x[..., s["rot"]:]
        if s["interleaved"]:
            a, b = rot[..., 0::2], rot[..., 1::2]
            out = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
        else:
            a, b = rot[..., :s["rot"] // 2], rot[..., s["rot"] // 2:]
            out = torch.cat([a * c - b * n, b * c + a * n], -1)
        return torch.cat([out, rest], -1)

    at = torch.arange(s["seq"], device="cuda")
    given = (at < s["counts"][:, None])[:, :, None, None]
    page, place = _place(s, s["lengths"][:, None] + at)
    k, v = _bits(s["k_cache"]), _bits(s["v_cache"])
    k[page, place] = torch.where(given, _bits(_coded(s, turn(s["k"]), K_SCALE)), k[page, place])
    v[page, place] = torch.where(given, _bits(_coded(s, s["v"].float(), V_SCALE)), v[page, place])
    q = torch.where(given, turn(s["q"]).to(s["out"].dtype), s["out"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _seen(s):
    """[batch, new token, entry]: whether the token sees the entry."""
    b, n = s["batch"], s["seq"]
    entry = torch.arange(s["pages"].shape[1] * s["page"], device="cuda")
    new = entry - s["lengths"][:, None]  # which of the new tokens the entry is
    token = torch.arange(n, device="cuda")
    if s["mask"] is None:
        ok = new[:, None] <= token[:, None]
    else:
        row = new.clamp(0, n - 1)[:, None].expand(b, n, -1)
        words = torch.gather(s["mask"], 2, row >> 5)
        ok = (new[:, None] < 0) | (((words >> (row & 31).to(torch.int32)) & 1) != 0)
    return ok & (new < s["counts"][:, None])[:, None] & (token < s["counts"][:, None])[:, :, None]


def _gathered(s, cache, scale, dtype):
    """[batch, kv, entry, dim]"""
    c = _bits(cache)[s["pages"].long()].view(cache.dtype).to(dtype)
    c = c.flatten(1, 2).transpose(1, 2)
    return c * scale if s["cache"] == "f8" else c


def _plain_attend(s):
    b, n, h, kv, d = s["batch"], s["seq"], s["heads"], s["kv"], s["dim"]
    k, v = _gathered(s, s["k_cache"], K_SCALE, torch.float32), _gathered(s, s["v_cache"], V_SCALE, torch.float32)
    q = s["q"].float().view(b, n, kv, h // kv, d).permute(0, 2, 3, 1, 4).reshape(b, kv, h // kv * n, d)
    x = (q @ k.transpose(2, 3) * d ** -0.5).view(b, kv, h // kv, n, -1)
    x = torch.where(_seen(s)[:, None, None], x, torch.full((), -math.inf, device="cuda"))
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    o = (e.view(b, kv, h // kv * n, -1) @ v).view(b, kv, h // kv, n, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).permute(0, 3, 1, 2, 4).reshape(b, n, h, d)
    given = torch.arange(n, device="cuda") < s["counts"][:, None]
    got = {"out": torch.where(given[:, :, None, None], o.to(s["out"].dtype), s["out"])}
    if s["lse"]:
        lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(b, n, h)
        got["lse"] = torch.where(given[:, :, None], lse, s["stats"])
    return got


def _plain_accept(s):
    b, n = s["batch"], s["seq"]
    node = torch.arange(n, dtype=torch.int32, device="cuda")
    up = s["parents"].clamp(min=0).long()
    right = (s["tokens"] == torch.gather(s["picks"], 1, up)) & (node > 0)
    # of siblings with the right token, the first
    same = (s["parents"][:, :, None] == s["parents"][:, None]) & right[:, None] & (node < node[:, None])
    right = (right & ~same.any(-1)) | (node == 0)
    taken = ~(s["above"] & ~right[:, None]).any(-1)  # a node all of whose way up is right
    path = torch.where(taken, node, n).sort(1).values
    accepted = taken.sum(1, dtype=torch.int32)
    last = torch.gather(path, 1, accepted[:, None].long() - 1)
    path = torch.where(path < n, path, -1)
    source = torch.where(path < 0, node, path)
    here, there = _place(s, s["lengths"][:, None] + source), _place(s, s["lengths"][:, None] + node)
    for c in (_bits(s["k_cache"]), _bits(s["v_cache"])):
        c[:, there[0], there[1]] = c[:, here[0], here[1]]
    return {"path": path, "accepted": accepted, "next": torch.gather(s["picks"], 1, last.long())[:, 0],
            "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# ---- the framework's entry points --------------------------------------------------------------------------
def _own_run(s):
    import transpose_heroes_gb300 as hf

    scales = dict(k_scale=K_SCALE, v_scale=V_SCALE) if s["cache"] == "f8" else {}
    if s["op"] == "append":
        hf.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["pages"], s["lengths"], counts=s["counts"], q=s["q"],
                        q_out=s["out"], positions=s["positions"], turns=s["turns"], interleaved=s["interleaved"], **scales)
        return {"q": s["out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["op"] == "attend":
        if s["ws"] is None:  # the scratch of a serving program, allocated once
            size = hf.cache_attention_workspace_size(s["batch"], s["seq"], s["heads"], s["kv"], s["dim"])
            s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        hf.cache_attention(s["q"], s["k_cache"], s["v_cache"], s["pages"], s["lengths"], s["out"], counts=s["counts"], mask=s["mask"],
                           lse=s["stats"], workspace=s["ws"], **scales)
        return {"out": s["out"], "lse": s["stats"]} if s["lse"] else {"out": s["out"]}
    hf.tree_accept(s["tokens"], s["parents"], s["picks"], s["path"], s["accepted"], s["next"], counts=s["counts"],
                   k_cache=s["k_cache"], v_cache=s["v_cache"], pages=s["pages"], lengths=s["lengths"])
    return {"path": s["path"], "accepted": s["accepted"], "next": s["next"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def run(s):
    if own:
        return _own_run(s)
    return {"append": _plain_append, "attend": _plain_attend, "accept": _plain_accept}[s["op"]](s)


# ---- what a pass cannot do without ---------------------------------------------------------------------------
def work(case):
    op, b = case["op"], case["batch"]
    c = EB[case["cache"]]
    if op == "accept":
        moved = sum(k - 1 for k in _kept(case))
        return {"bytes": moved * 4 * case["layers"] * case["kv"] * case["dim"] * c + b * (case["seq"] * 16 + 12), "flops": 0}
    e, h, kv, d = EB[case["dtype"]], case["heads"], case["kv"], case["dim"]
    counts, lengths = _counts(case), _lengths(case)
    tokens = sum(counts)
    if op == "append":
        return {"bytes": tokens * d * (2 * h * e + 2 * kv * (e + c)) + tokens * 4, "flops": tokens * (h + kv) * case["rot"] * 3}
    entries = sum(lengths) + tokens
    if case["tree"]:
        pairs = sum(n * (sum(lengths) / b + n) for n in counts)
    else:
        pairs = sum(n * (sum(lengths) / b + (n + 1) / 2) for n in counts)
    side = tokens * ((case["seq"] + 31) // 32 * 4 if case["tree"] else 0) + (tokens * h * 4 if case["lse"] else 0)
    return {"bytes": 2 * tokens * h * d * e + 2 * entries * kv * d * c + side, "flops": 4 * h * d * pairs}


# ---- the operators in 64 bits ----------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "accept":
        return None  # whole numbers, and entries that are copied
    s = prepare(case, seed)
    b, n, h, kv, d = s["batch"], s["seq"], s["heads"], s["kv"], s["dim"]
    lengths, counts = s["lengths"].tolist(), s["counts"].tolist()
    if s["op"] == "append":
        pair = torch.arange(s["rot"] // 2, dtype=torch.float64, device="cuda")
        angle = _positions(s).double()[..., None] * 10000.0 ** (-2.0 * pair / s["rot"])
        z = torch.polar(torch.ones_like(angle), angle)[:, :, None]
        half = s["rot"] // 2
        first, second = (slice(0, s["rot"], 2), slice(1, s["rot"], 2)) if s["interleaved"] else (slice(0, half), slice(half, s["rot"]))

        def turned(x):
            x = x.double()
            w = torch.complex(x[..., first], x[..., second]) * z
            x[..., first], x[..., second] = w.real, w.imag
            return x

        q, k, v = turned(s["q"]), turned(s["k"]), s["v"].double()
        if s["cache"] == "f8":
            k, v = (k / K_SCALE).clamp(-F8_MAX, F8_MAX), (v / V_SCALE).clamp(-F8_MAX, F8_MAX)
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        for i in range(b):
            slot = torch.arange(lengths[i], lengths[i] + counts[i], device="cuda")
            page = s["pages"][i].long()[slot.div(s["page"], rounding_mode="floor")]
            kc[page, slot % s["page"]], vc[page, slot % s["page"]] = k[i, :counts[i]], v[i, :counts[i]]
            q[i, counts[i]:] = 0.0
        return {"q": q, "k_cache": kc, "v_cache": vc}
    if sum((lengths[i] + counts[i]) * counts[i] for i in range(b)) * h * d > 1 << 42:
        return None
    out = torch.zeros(b, n, h, d, dtype=torch.float64, device="cuda")
    stats = torch.zeros(b, n, h, dtype=torch.float64, device="cuda")
    for i in range(b):
        total, new = lengths[i] + counts[i], counts[i]
        slot = torch.arange(total, device="cuda")
        page, place = s["pages"][i].long()[slot.div(s["page"], rounding_mode="floor")], slot % s["page"]
        k, v = (_bits(c)[page, place].view(c.dtype).double().repeat_interleave(h // kv, 1) for c in (s["k_cache"], s["v_cache"]))
        if s["cache"] == "f8":
            k, v = k * K_SCALE, v * V_SCALE
        hidden = torch.zeros(new, total, dtype=torch.bool, device="cuda")
        hidden[:, lengths[i]:] = ~s["above"][i, :new, :new] if s["tree"] else torch.ones(new, new, device="cuda").triu(1).bool()
        x = torch.einsum("thd,shd->hts", s["q"][i, :new].double(), k) / math.sqrt(d)
        x.masked_fill_(hidden, -math.inf)
        stats[i, :new] = torch.logsumexp(x, -1).T
        out[i, :new] = torch.einsum("hts,shd->thd", x.softmax(-1), v)
    return {"out": out, "lse": stats} if s["lse"] else {"out": out}
