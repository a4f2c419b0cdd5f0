"""The paged cache's operators on the GPU against their 64-bit statements (tests/cache_reference.py)."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import cache_reference as ref
import transpose_heroes_gb300 as hf
from layer_reference import HALF_ULP

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transpose_heroes_gb300 import build

    build.build()
    hf.lib()


def workspace(q, kv):
    return torch.empty(hf.cache_attention_workspace_size(*q.shape[:3], kv, q.shape[3]), dtype=torch.uint8, device=DEV).fill_(0xFF)


# ---- attention -------------------------------------------------------------------------------------------------
def attend(rng, lengths, counts, seq, heads, kv, dim, page, dtype="bf16", cache=None, tree="causal", std=1.0, scale=None, one_tree=False,
           q_layout="packed", change=None, check=True, **kw):
    """Runs one case and holds out and lse to their bounds. tree: "causal", "tree" (random trees) or "random" bits."""
    cache = cache or dtype
    scales = dict(k_scale=0.02, v_scale=0.015) if cache == "f8" else {}
    c = ref.filled(rng, lengths, counts, seq, kv, dim, page, cache, DEV, **scales, **kw)
    b = len(lengths)
    if q_layout == "packed":
        q = ref.normal(rng, (b, seq, heads + 3, dim), dtype, std).to(DEV)[:, :, 1:1 + heads]
    elif q_layout == "heads":
        q = ref.normal(rng, (b, heads, seq, dim), dtype, std).to(DEV).transpose(1, 2)
    else:
        q = ref.normal(rng, (b, seq, heads, dim + 3), dtype, std).to(DEV)[..., 1:1 + dim]
    sees = np.tril(np.ones((b, seq, seq), bool))
    mask = None
    if tree != "causal":
        for i in range(b):
            sees[i] = sees[0] if one_tree and i else ref.sees_of(ref.random_tree(rng, seq)) if tree == "tree" else rng.random((seq, seq)) < 0.4
        mask = ref.packed(sees).to(DEV)
    if change:
        change(c, sees)
    out = torch.full((b, seq, heads, dim + 5), 7.0, dtype=ref.DT[dtype], device=DEV)
    view = out[..., 2:2 + dim] if q_layout != "packed" else out[..., :dim]
    lse = torch.full((b, seq, heads), 7.0, device=DEV)
    got = hf.cache_attention(q, c.k, c.v, c.table, c.len, view, counts=torch.tensor(counts, dtype=torch.int32, device=DEV), mask=mask,
                             scale=scale, lse=lse, workspace=workspace(q, kv), **scales)
    assert got is view
    torch.cuda.synchronize()
    edge = out.clone()
    (edge[..., 2:2 + dim] if q_layout != "packed" else edge[..., :dim]).fill_(7.0)
    assert bool((edge == 7.0).all())
    if not check:
        return c, q, view, lse, sees
    weights = None if dtype == "f32" else "f16" if cache == "f8" else dtype
    for i in range(b):
        n, m = lengths[i], counts[i]
        assert bool((view[i, m:] == 7.0).all()) and bool((lse[i, m:] == 7.0).all())
        if not m:
            continue
        k, v = c.get(i, range(n + m))
        full = np.concatenate([np.ones((m, n), bool), sees[i, :m, :m]], 1)
        want, wlse, bound, elen = ref.attention(q[i, :m].double().cpu(), k, v, full, scale or dim ** -0.5)
        err = (view[i, :m].double().cpu() - want).abs()
        limit = bound(weights) + ref.rounding(want, dtype) * (1 + 2.0 ** -6)
        assert bool((err <= limit).all()), (i, float((err / limit).max()), np.argwhere(~(err <= limit).numpy())[:4])
        g = lse[i, :m].double().cpu()
        none = torch.isinf(wlse)
        assert bool((g[none] == -math.inf).all())
        assert bool(((g - wlse).abs() <= elen)[~none].all()), float((g - wlse).abs()[~none].max())
    return c, q, view, lse, sees


TYPES = [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f8"), ("f16", "f8"), ("f32", "f8")]


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
def test_single_tokens(dtype, cache, dim):
    attend(np.random.default_rng(1), [0, 1, 17, 63, 64, 65, 200, 511], [1] * 8, 1, 8, 2, dim, 16, dtype, cache)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("tree", ["causal", "tree", "random"])
def test_trees(dtype, cache, tree):
    attend(np.random.default_rng(2), [0, 5, 100, 255, 31], [7, 12, 1, 0, 12], 12, 8, 2, 128, 16, dtype, cache, tree)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("tree", ["causal", "tree"])
def test_large_trees(dtype, cache, tree):
    """More rows than one tile: 70 tokens of 4 heads."""
    attend(np.random.default_rng(3), [0, 300, 129, 127], [70, 33, 64, 70], 70, 8, 2, 128, 32, dtype, cache, tree)


@pytest.mark.parametrize("dim", [1, 8, 40, 50, 72, 80, 96, 112, 160, 192, 256])
@pytest.mark.parametrize("dtype,cache", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f8")])
def test_head_sizes(dim, dtype, cache):
    attend(np.random.default_rng(dim), [3, 77, 150], [3, 5, 1], 5, 6, 3, dim, 16, dtype, cache, "tree")
    attend(np.random.default_rng(dim), [3, 150], [40, 37], 40, 6, 3, dim, 16, dtype, cache, "causal")


@pytest.mark.parametrize("page", [1, 2, 5, 7, 16, 24, 100, 128, 300])
@pytest.mark.parametrize("dtype,cache,seq", [("bf16", "bf16", 2), ("bf16", "bf16", 50), ("f16", "f8", 3), ("f16", "f8", 41), ("f32", "f32", 4)])
def test_page_sizes(page, dtype, cache, seq):
    attend(np.random.default_rng(page), [0, 33, 130, 257], [seq, seq - 1, 1, seq], seq, 4, 1, 64, page, dtype, cache, "tree")


@pytest.mark.parametrize("heads,kv", [(1, 1), (7, 1), (8, 8), (14, 2), (32, 8), (64, 4), (40, 1), (300, 2)])
@pytest.mark.parametrize("dtype,seq", [("bf16", 1), ("bf16", 9), ("f16", 33), ("f32", 3)])
def test_groups(heads, kv, dtype, seq):
    attend(np.random.default_rng(heads), [0, 70, 200], [seq, seq, 1], seq, heads, kv, 64, 16, dtype, None, "tree")


@pytest.mark.parametrize("layout", ["packed", "heads", "odd"])
@pytest.mark.parametrize("major,pad", [(False, 0), (True, 0), (False, 8), (True, 3)])
@pytest.mark.parametrize("seq", [2, 45])
def test_strides(layout, major, pad, seq):
    attend(np.random.default_rng(5), [10, 140], [seq, seq - 1], seq, 8, 2, 64, 16, "bf16", None, "tree", q_layout=layout, heads_major=major,
           pad=pad)


@pytest.mark.parametrize("dtype,cache,seq", [("bf16", "bf16", 1), ("bf16", "bf16", 40), ("f16", "f8", 2), ("f16", "f8", 40), ("f32", "f32", 1)])
def test_long_contexts(dtype, cache, seq):
    """One long sequence among short ones: its work is shared by many blocks."""
    attend(np.random.default_rng(6), [20000, 3, 900], [seq, 1, seq], seq, 8, 2, 128, 64, dtype, cache, "causal")
    attend(np.random.default_rng(7), [7001], [seq], seq, 4, 1, 64, 16, dtype, cache, "tree", std=3.0)


def test_prompts():
    attend(np.random.default_rng(8), [0, 100], [700, 523], 700, 8, 2, 128, 64, "bf16")
    attend(np.random.default_rng(9), [0, 1000, 5], [300, 511, 130], 511, 4, 1, 64, 16, "f16")
    attend(np.random.default_rng(10), [0, 77], [300, 200], 300, 4, 2, 128, 16, "bf16", "f8")
    attend(np.random.default_rng(10), [0, 77], [130, 200], 200, 4, 2, 64, 16, "f32")


def test_many_sequences():
    rng = np.random.default_rng(11)
    n = 700
    attend(rng, [int(x) for x in rng.integers(0, 40, n)], [int(x) for x in rng.integers(0, 3, n)], 2, 4, 2, 64, 16, "bf16")


@pytest.mark.parametrize("dtype,cache,page", [("bf16", "bf16", 16), ("f16", "f16", 7), ("bf16", "f8", 16), ("f32", "f32", 16)])
def test_masks_of_several_tiles(dtype, cache, page):
    """Trees and arbitrary masks wider than a tile of entries, whose words begin anywhere in it."""
    for tree in ("tree", "random"):
        attend(np.random.default_rng(50), [100, 7, 0], [300, 211, 129], 300, 4, 2, 64, page, dtype, cache, tree)


@pytest.mark.parametrize("dtype,cache,page", [("bf16", "bf16", 16), ("f16", "f16", 5), ("bf16", "f8", 16), ("f32", "f32", 8)])
@pytest.mark.parametrize("tree", ["causal", "tree"])
def test_tokens_that_have_no_room(dtype, cache, page, tree):
    """New tokens behind the table's pages are seen by nobody, and see what is there."""
    rng = np.random.default_rng(51)
    seq, n = 40, 150
    c = ref.filled(rng, [n], [seq], seq, 2, 64, page, cache, DEV)
    room = c.width - -(-25 // page)  # pages: some of the new tokens are left out
    cap = room * page
    q = ref.normal(rng, (1, seq, 8, 64), dtype).to(DEV)
    sees = np.tril(np.ones((seq, seq), bool)) if tree == "causal" else ref.sees_of(ref.random_tree(rng, seq))
    mask = None if tree == "causal" else ref.packed(sees).to(DEV)
    for length in (n, cap - 3, cap, cap + 100):
        out, lse = torch.empty_like(q), torch.empty(1, seq, 8, device=DEV)
        hf.cache_attention(q, c.k, c.v, c.table[:, :room], torch.tensor([length], dtype=torch.int32, device=DEV), out, mask=mask, lse=lse,
                           workspace=workspace(q, 2))
        old = min(length, cap)
        k, v = c.get(0, range(cap))
        full = np.concatenate([np.ones((seq, old), bool), sees], 1)[:, :cap]
        want, wlse, bound, elen = ref.attention(q[0].double().cpu(), k, v, full, 0.125)
        weights = None if dtype == "f32" else "f16" if cache == "f8" else dtype
        assert bool(((out[0].double().cpu() - want).abs() <= bound(weights) + 2 * ref.rounding(want, dtype)).all())
        assert bool(((lse[0].double().cpu() - wlse).abs() <= elen).all())


@pytest.mark.parametrize("page", [16, 5])
def test_many_sequences_of_many_rows(page):
    rng = np.random.default_rng(52)
    n = 560
    attend(rng, [int(x) for x in rng.integers(0, 60, n)], [int(x) for x in rng.integers(0, 18, n)], 17, 4, 2, 64, page, "bf16")


@pytest.mark.parametrize("dtype,cache,seq", [("bf16", "bf16", 4), ("bf16", "bf16", 40), ("f16", "f8", 4), ("f16", "f8", 40), ("f32", "f32", 4)])
def test_sharp_weights_and_far_maxima(dtype, cache, seq):
    """Scores of many hundreds: the running maximum moves often and far."""
    attend(np.random.default_rng(12), [600, 130], [seq, 1], seq, 8, 2, 64, 16, dtype, cache, "tree", std=30.0)
    attend(np.random.default_rng(13), [600, 130], [seq, 1], seq, 8, 2, 64, 16, dtype, cache, "tree", scale=1e-3)


def test_one_tree_for_all():
    attend(np.random.default_rng(14), [5, 60, 0], [9, 9, 9], 9, 4, 2, 64, 16, "bf16", None, "tree", one_tree=True)
    rng = np.random.default_rng(15)
    sees = ref.sees_of(ref.random_tree(rng, 40))
    c = ref.filled(rng, [33, 70], [40, 40], 40, 2, 64, 16, "bf16", DEV)
    q = ref.normal(rng, (2, 40, 4, 64), "bf16").to(DEV)
    outs = []
    for mask in (ref.packed(sees).to(DEV), ref.packed(np.stack([sees, sees])).to(DEV)):
        outs.append(hf.cache_attention(q, c.k, c.v, c.table, c.len, torch.empty_like(q), mask=mask, workspace=workspace(q, 2)))
    assert torch.equal(*outs)


def test_rows_that_see_nothing():
    """No entry before them and no bit of their own: 0 and -inf; the others as they are."""
    for seq in (3, 40):
        for dtype, cache in TYPES:
            def blank(c, sees):
                sees[:, 1] = False

            rng = np.random.default_rng(16)
            c = ref.filled(rng, [0, 4], [seq, seq], seq, 2, 64, 16, cache, DEV)
            sees = np.tril(np.ones((2, seq, seq), bool))
            sees[:, 1] = False
            q = ref.normal(rng, (2, seq, 4, 64), dtype).to(DEV)
            lse = torch.empty(2, seq, 4, device=DEV)
            out = hf.cache_attention(q, c.k, c.v, c.table, c.len, torch.empty_like(q), mask=ref.packed(sees).to(DEV), lse=lse,
                                     workspace=workspace(q, 2))
            assert bool((out[0, 1] == 0).all()) and bool((lse[0, 1] == -math.inf).all())
            assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse[1]).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype,cache,seq", [("bf16", "bf16", 6), ("bf16", "bf16", 60), ("f16", "f16", 60), ("f16", "f8", 6), ("bf16", "f8", 60),
                                             ("f32", "f32", 6)])
@pytest.mark.parametrize("page", [16, 7])
def test_what_is_not_seen_does_not_matter(page, bad, dtype, cache, seq):
    """A NaN or infinite key and value of one drafted node: only the rows that see it change."""
    if cache == "f8":
        bad = math.nan
    for tree in ("causal", "tree"):
        rng = np.random.default_rng(17)
        node = seq // 2
        runs = []
        for poison in (False, True):
            def change(c, sees):
                if poison:
                    for i, n in enumerate(c.lengths):
                        k, v = (torch.full((1, 2, 64), bad) for _ in range(2))
                        c.put(i, [n + node], k, v)

            runs.append(attend(np.random.default_rng(18), [0, 50, 130], [seq] * 3, seq, 8, 2, 64, page, dtype, cache, tree, change=change, check=False))
        (_, _, a, la, sees), (_, _, b, lb, _) = runs
        for i in range(3):
            unseen = torch.from_numpy(~sees[i, :, node])
            assert torch.equal(a[i][unseen], b[i][unseen]) and torch.equal(la[i][unseen], lb[i][unseen])
            assert not bool(torch.isfinite(b[i][~unseen]).all(-1).any())


@pytest.mark.parametrize("page", [5, 8, 128])
@pytest.mark.parametrize("dim", [64, 128])
def test_an_infinite_value_of_the_prompt(page, dim):
    """In entries that all rows see, beside and apart from tiles that a mask cuts: every row's element is infinite, and no other."""
    for seq, at in ((60, 3), (60, 139), (6, 3), (6, 149)):
        def change(c, sees):
            where = c.where(0, [at])
            c.v[where[0], where[1], 1, 7] = -math.inf

        clean = attend(np.random.default_rng(60), [150], [seq], seq, 4, 2, dim, page, "bf16", None, "tree")
        dirty = attend(np.random.default_rng(60), [150], [seq], seq, 4, 2, dim, page, "bf16", None, "tree", change=change, check=False)
        want = clean[2][0].clone()
        want[:, 2:, 7] = -math.inf
        assert torch.equal(dirty[2][0], want)


@pytest.mark.parametrize("dtype,cache,seq", [("bf16", "bf16", 6), ("bf16", "bf16", 60), ("f16", "f8", 6), ("f16", "f8", 60), ("f32", "f32", 6)])
def test_an_infinite_value_among_finite_keys(dtype, cache, seq):
    """Only the elements whose own value is infinite or NaN change, in the rows that see it."""
    node = 2

    def change(c, sees):
        page, place = c.where(0, [c.lengths[0] + node])
        c.raw(c.v)[page, place, 0, 5] = c.raw(torch.tensor([math.nan if cache == "f8" else math.inf]).to(ref.DT[cache]).to(DEV))

    clean = attend(np.random.default_rng(19), [40], [seq], seq, 4, 2, 64, 16, dtype, cache, "tree")
    dirty = attend(np.random.default_rng(19), [40], [seq], seq, 4, 2, 64, 16, dtype, cache, "tree", change=change, check=False)
    sees = torch.from_numpy(clean[4][0, :, node])
    want = clean[2][0].clone()
    hit = torch.zeros(want.shape, dtype=torch.bool)
    hit[sees, :2, 5] = True
    hit = hit.to(DEV)
    got = dirty[2][0]
    assert torch.equal(got[~hit], want[~hit]) and not bool(torch.isfinite(got[hit]).any())


@pytest.mark.parametrize("dtype,cache,seq", [("bf16", "bf16", 2), ("bf16", "bf16", 40), ("f16", "f8", 2), ("f16", "f8", 40), ("f32", "f32", 2)])
def test_pages_that_are_not_there(dtype, cache, seq):
    """Entries in a page outside the cache are seen by nobody."""
    rng = np.random.default_rng(20)
    c = ref.filled(rng, [200], [seq], seq, 2, 64, 16, cache, DEV)
    q = ref.normal(rng, (1, seq, 4, 64), dtype).to(DEV)
    for bad in (-1, c.total, 2 ** 31 - 1, -2 ** 31):
        table = c.table.clone()
        table[0, 3] = table[0, 7] = bad
        out, lse = torch.empty_like(q), torch.empty(1, seq, 4, device=DEV)
        hf.cache_attention(q, c.k, c.v, table, c.len, out, lse=lse, workspace=workspace(q, 2))
        k, v = c.get(0, range(200 + seq))
        sees = np.concatenate([np.ones((seq, 200), bool), np.tril(np.ones((seq, seq), bool))], 1)
        sees[:, 48:64] = sees[:, 112:128] = False
        want, wlse, bound, elen = ref.attention(q[0].double().cpu(), k, v, sees, 64 ** -0.5)
        weights = None if dtype == "f32" else "f16" if cache == "f8" else dtype
        assert bool(((out[0].double().cpu() - want).abs() <= bound(weights) + 2 * ref.rounding(want, dtype)).all())
        assert bool(((lse[0].double().cpu() - wlse).abs() <= elen).all())


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("seq", [1, 40])
def test_a_cache_without_pages(dtype, cache, seq):
    """Nothing can be written to it, and nobody sees anything."""
    c = [torch.empty(0, 16, 2, 64, dtype=ref.DT[cache], device=DEV) for _ in range(2)]
    q = ref.normal(np.random.default_rng(1), (2, seq, 4, 64), dtype).to(DEV)
    for width in (0, 3):
        table, lengths = torch.zeros(2, width, dtype=torch.int32, device=DEV), torch.tensor([0, 20], dtype=torch.int32, device=DEV)
        lse = torch.zeros(2, seq, 4, device=DEV)
        hf.cache_append(q[:, :, :2], q[:, :, 2:], *c, table, lengths)
        out = hf.cache_attention(q, *c, table, lengths, torch.full_like(q, 7.0), lse=lse, workspace=workspace(q, 2))
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_lengths_outside_the_cache():
    """Clamped: negative lengths are 0, and entries behind the table's pages are seen by nobody."""
    rng = np.random.default_rng(21)
    c = ref.filled(rng, [62], [2], 2, 2, 64, 16, "bf16", DEV)
    q = ref.normal(rng, (1, 2, 4, 64), "bf16").to(DEV)

    def run(length, counts=None):
        return hf.cache_attention(q, c.k, c.v, c.table, torch.tensor([length], dtype=torch.int32, device=DEV), torch.full_like(q, 7.0),
                                  counts=None if counts is None else torch.tensor([counts], dtype=torch.int32, device=DEV), workspace=workspace(q, 2))

    k, v = c.get(0, range(64))

    def near(got, n, sees):
        want, _, bound, _ = ref.attention(q[0].double().cpu(), k[:n], v[:n], sees, 0.125)
        assert bool(((got[0].double().cpu() - want).abs() <= bound("bf16") + 2 * ref.rounding(want, "bf16")).all())

    near(run(2 ** 31 - 1), 64, np.ones((2, 64), bool))
    near(run(63), 64, np.ones((2, 64), bool))
    near(run(-5), 2, np.tril(np.ones((2, 2), bool)))
    assert bool((run(62, -3) == 7.0).all())
    near(run(62, 9), 64, np.tril(np.ones((2, 64), bool), 62))


def test_in_place_and_the_same_twice():
    for seq, n in ((1, 3000), (50, 700)):
        rng = np.random.default_rng(22)
        c = ref.filled(rng, [n, 10], [seq, seq], seq, 2, 128, 16, "bf16", DEV)
        q = ref.normal(rng, (2, seq, 8, 128), "bf16").to(DEV)
        a = hf.cache_attention(q, c.k, c.v, c.table, c.len, torch.empty_like(q), workspace=workspace(q, 2))
        b = hf.cache_attention(q, c.k, c.v, c.table, c.len, torch.empty_like(q), workspace=workspace(q, 2).zero_())
        assert torch.equal(a, b)
        hf.cache_attention(q, c.k, c.v, c.table, c.len, q, workspace=workspace(q, 2))
        assert torch.equal(a, q)


# ---- appending ---------------------------------------------------------------------------------------------------
def append(rng, lengths, counts, seq, heads, kv, dim, rot, page, dtype="bf16", cache=None, interleaved=False, positions=None, scale=1.0,
           q_inplace=False, pad=0, **kw):
    cache = cache or dtype
    scales = dict(k_scale=0.02, v_scale=0.015) if cache == "f8" else {}
    c = ref.filled(rng, lengths, [0] * len(lengths), seq, kv, dim, page, cache, DEV, pad=pad, **scales, **kw)
    before = [c.raw(s).clone() for s in c.stores]
    b = len(lengths)
    qkv = ref.normal(rng, (b, seq, heads + 2 * kv, dim + pad), dtype).to(DEV)[..., :dim]
    q, k, v = qkv[:, :, :heads], qkv[:, :, heads:heads + kv], qkv[:, :, heads + kv:]
    words = hf.rotary_turns(rot)
    turns = torch.from_numpy(words).to(DEV) if rot else None
    at = np.array(lengths)[:, None] + np.arange(seq) if positions is None else positions
    pos = None if positions is None else torch.from_numpy(at.astype(np.int32)).to(DEV)
    q0 = q.double().cpu()
    out = q if q_inplace else torch.full((b, seq, heads, dim), 7.0, dtype=ref.DT[dtype], device=DEV)
    hf.cache_append(k, v, c.k, c.v, c.table, c.len, counts=torch.tensor(counts, dtype=torch.int32, device=DEV), q=q if heads else None,
                    q_out=out if heads else None, positions=pos, turns=turns, interleaved=interleaved, scale=scale, **scales)
    torch.cuda.synchronize()
    after = [c.raw(s).clone() for s in c.stores]
    for i in range(b):
        m = counts[i]
        tq, eq = ref.turned(q0[i, :m], at[i, :m], words, interleaved, scale)
        assert bool(((out[i, :m].double().cpu() - tq).abs() <= eq + ref.rounding(tq.abs() + eq, dtype)).all())
        assert torch.equal(out[i, m:].double().cpu(), q0[i, m:] if q_inplace else torch.full_like(q0[i, m:], 7.0))
        if not m:
            continue
        tk, ek = ref.turned(k[i, :m].double().cpu(), at[i, :m], words, interleaved, scale)
        gk, gv = c.get(i, range(lengths[i], lengths[i] + m))
        ks, vs = c.k_scale, c.v_scale
        tv = v[i, :m].double().cpu()
        assert bool(((gk - tk).abs() / ks <= ek / ks + ref.rounding((tk.abs() + ek) / ks, cache) * (1 + 2.0 ** -20)).all())
        if cache == "f8":  # the quotient is rounded to f32 first
            assert bool(((gv - tv).abs() / vs <= ref.rounding(tv / vs, cache) * (1 + 2.0 ** -20)).all())
        else:
            assert torch.equal(gv, tv)
        page_, place = c.where(i, range(lengths[i], lengths[i] + m))
        for s in (c.k, c.v):  # what was written, as it was: nothing else changed
            c.raw(s)[page_, place] = 0x7F if cache == "f8" else math.nan
    for s, old in zip(c.stores, before):
        new = c.raw(s)
        assert torch.equal(new.view(torch.uint8) if new.dtype != torch.uint8 else new, old.view(torch.uint8) if old.dtype != torch.uint8 else old) or \
            bool(((new == old) | (torch.isnan(new.float()) & torch.isnan(old.float()))).all())


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(dtype, cache, interleaved):
    append(np.random.default_rng(30), [0, 5, 100, 16], [1, 1, 1, 0], 1, 8, 2, 128, 128, 16, dtype, cache, interleaved)
    append(np.random.default_rng(31), [0, 5, 100], [7, 3, 0], 7, 8, 2, 64, 32, 16, dtype, cache, interleaved, heads_major=True)


@pytest.mark.parametrize("dim,rot", [(1, 0), (2, 2), (8, 8), (40, 40), (50, 20), (80, 64), (96, 96), (256, 128), (512, 512), (33, 30)])
@pytest.mark.parametrize("dtype,cache", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f8")])
def test_append_head_sizes(dim, rot, dtype, cache):
    for inter in (False, True):
        append(np.random.default_rng(dim), [3, 77], [3, 5], 5, 3, 1, dim, rot, 7, dtype, cache, inter, pad=3 if dim == 40 else 0)


def test_append_many_tokens():
    append(np.random.default_rng(32), [0, 3], [900, 1000], 1000, 8, 2, 128, 128, 64, "bf16")
    append(np.random.default_rng(33), [0, 3], [900, 1000], 1000, 8, 2, 128, 64, 64, "bf16", "f8", True)
    append(np.random.default_rng(33), [0, 3], [300, 400], 400, 8, 4, 64, 64, 10, "f32", "f8", True)
    append(np.random.default_rng(34), [17] * 300, [1] * 300, 1, 32, 8, 128, 128, 16, "f16")


def test_append_positions_of_a_tree():
    rng = np.random.default_rng(35)
    _, depths = hf.tree_mask([-1, 0, 0, 1, 1, 2, 5])
    lengths = [9, 60]
    append(rng, lengths, [7, 7], 7, 4, 2, 64, 64, 16, positions=np.array(lengths)[:, None] + depths[None])
    append(rng, lengths, [7, 5], 7, 4, 2, 64, 64, 16, positions=np.array([[-3, 0, 2 ** 31 - 1, 5, 100000, 7, -2 ** 31]] * 2), scale=0.7)


def test_append_without_queries_and_in_place():
    append(np.random.default_rng(36), [4, 5], [2, 1], 2, 0, 2, 64, 64, 16)
    append(np.random.default_rng(37), [4, 5], [2, 1], 2, 4, 2, 64, 64, 16, q_inplace=True)


def test_append_drops_what_has_no_place():
    rng = np.random.default_rng(38)
    c = ref.Cache(rng, [14, 14, 14], 4, 2, 64, 16, "bf16", DEV)
    k = ref.normal(rng, (3, 4, 2, 64), "bf16").to(DEV)
    table = c.table.clone()
    table[0, 1], table[1, 1] = -1, c.total
    long = torch.tensor([14, 14, 2 * 16 - 1], dtype=torch.int32, device=DEV)
    hf.cache_append(k, k, c.k, c.v, table, long)
    torch.cuda.synchronize()
    for i, kept in ((0, 2), (1, 2), (2, 1)):
        page, place = c.where(i, range(int(long[i]), int(long[i]) + kept))
        assert torch.equal(c.k[page, place], k[i, :kept]) and torch.equal(c.v[page, place], k[i, :kept])
        c.k[page, place] = c.v[page, place] = math.nan
    assert bool(c.k.isnan().all()) and bool(c.v.isnan().all())


def test_append_codes_saturate_and_keep_nan():
    rng = np.random.default_rng(39)
    c = ref.Cache(rng, [0], 1, 1, 64, 16, "f8", DEV)
    k = torch.zeros(1, 1, 1, 64, device=DEV)
    k[..., 0], k[..., 1], k[..., 2], k[..., 3] = math.nan, math.inf, -1e30, 1e-30
    hf.cache_append(k, k, c.k, c.v, c.table, c.len, k_scale=0.5, v_scale=2.0)
    got = c.k[c.table[0, 0].long(), 0, 0].float()
    assert math.isnan(float(got[0])) and float(got[1]) == 448 and float(got[2]) == -448 and float(got[3]) == 0 and bool((got[4:] == 0).all())


# ---- acceptance ----------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("seq,batch", [(1, 3), (2, 2), (16, 5), (33, 40), (200, 7), (1500, 2), (4096, 1)])
@pytest.mark.parametrize("with_cache", [False, True])
def test_tree_accept(seq, batch, with_cache):
    rng = np.random.default_rng(seq)
    vocab = 4  # so that siblings often hold the same token
    tokens, picks = rng.integers(0, vocab, (batch, seq)), rng.integers(-1, vocab, (batch, seq))
    parents = np.array([ref.random_tree(rng, seq) for _ in range(batch)])
    parents[:, 0] = rng.integers(-2, seq, batch)  # does not matter
    for i in range(batch):
        for c in range(1, seq):  # long chains in some
            if i % 2 and rng.random() < 0.7:
                parents[i, c] = c - 1
                picks[i, c - 1] = tokens[i, c]
            elif rng.random() < 0.05:
                parents[i, c] = rng.integers(c, seq + 5)  # not before it: nobody's child
    counts = rng.integers(0, seq + 1, batch)
    counts[0] = seq
    lengths = [int(x) for x in rng.integers(0, 30, batch)]
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)  # noqa: E731
    path, accepted, nxt = (torch.full(s, 77, dtype=torch.int32, device=DEV) for s in ((batch, seq), (batch,), (batch,)))
    kw = {}
    if with_cache:
        c = ref.filled(rng, lengths, [seq] * batch, seq, 2, 20, 7, "f16", DEV, layers=3)
        old = [t.clone() for t in (c.k, c.v)]
        kw = dict(k_cache=c.k, v_cache=c.v, pages=c.table, lengths=c.len)
    hf.tree_accept(dev(tokens), dev(parents), dev(picks), path, accepted, nxt, counts=dev(counts), **kw)
    torch.cuda.synchronize()
    for i in range(batch):
        want = ref.accept(tokens[i], parents[i], picks[i], counts[i])
        assert int(accepted[i]) == len(want)
        assert path[i].tolist() == want + [-1] * (seq - len(want))
        assert int(nxt[i]) == (picks[i][want[-1]] if want else -1)
        if with_cache and want:
            src, dst = c.where(i, [lengths[i] + x for x in want]), c.where(i, range(lengths[i], lengths[i] + len(want)))
            for o in old:
                o[:, dst[0], dst[1]] = o[:, src[0], src[1]]
    if with_cache:
        for o, t in zip(old, (c.k, c.v)):
            assert torch.equal(o.view(torch.int16), t.view(torch.int16))


@pytest.mark.parametrize("dtype,dim,major,pad", [("bf16", 64, False, 0), ("bf16", 64, True, 0), ("f8", 64, False, 0), ("f8", 9, False, 0), ("f32", 3, True, 1),
                                                 ("f16", 12, False, 0), ("bf16", 33, False, 2)])
def test_accepted_entries_of_any_size(dtype, dim, major, pad):
    """A chain that skips nodes, over pages that end inside it; one layer, given without a dimension of layers."""
    rng = np.random.default_rng(dim)
    seq, lengths = 20, [3, 14]
    chain = [0, 1, 4, 9, 10, 15, 19]
    parents = np.zeros((2, seq), np.int32)
    tokens, picks = np.tile(np.arange(seq), (2, 1)), np.full((2, seq), 1000)
    for a, b in zip(chain, chain[1:]):
        parents[:, b], picks[:, a] = a, b
    c = ref.filled(rng, lengths, [seq] * 2, seq, 3, dim, 5, dtype, DEV, heads_major=major, pad=pad)
    old = [c.raw(t).clone() for t in (c.k, c.v)]
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)  # noqa: E731
    path, accepted, nxt = torch.empty(2, seq, dtype=torch.int32, device=DEV), dev([0, 0]), dev([0, 0])
    bad = c.table.clone()
    bad[1, (14 + 10) // 5] = -1  # the page of node 10: it stays where it is
    hf.tree_accept(dev(tokens), dev(parents[0]), dev(picks), path, accepted, nxt, k_cache=c.k, v_cache=c.v, pages=bad, lengths=c.len)
    assert accepted.tolist() == [7, 7] and nxt.tolist() == [1000, 1000]
    for i in range(2):
        for to, node in enumerate(chain):
            gone = i == 1 and ((14 + node) // 5 == 24 // 5 or (14 + to) // 5 == 24 // 5)
            if to == node or gone:
                continue
            s, d = c.where(i, [lengths[i] + node]), c.where(i, [lengths[i] + to])
            for o in old:
                o[d[0], d[1]] = o[s[0], s[1]]
    for o, t in zip(old, (c.k, c.v)):
        a, b = o.contiguous(), c.raw(t).contiguous()
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ---- together --------------------------------------------------------------------------------------------------------
def test_append_attend_and_accept_in_a_captured_step():
    """One captured step, replayed while lengths move: what a serving loop does. Two graphs share the workspace, one after another."""
    rng = np.random.default_rng(40)
    b, seq, heads, kv, dim, page = 2, 5, 4, 2, 64, 16
    c = ref.filled(rng, [30, 7], [0, 0], 40, kv, dim, page, "bf16", DEV)
    parents = [-1, 0, 0, 2, 1]
    mask, depths = (torch.from_numpy(x).to(DEV) for x in hf.tree_mask(parents))
    up = torch.tensor(parents, dtype=torch.int32, device=DEV)
    turns = torch.from_numpy(hf.rotary_turns(dim)).to(DEV)
    qkv = ref.normal(rng, (b, seq, heads + 2 * kv, dim), "bf16").to(DEV)
    tokens = torch.arange(seq, dtype=torch.int32, device=DEV).repeat(b, 1)
    picks = torch.tensor([[2, 9, 3, 8, 9], [1, 4, 9, 9, 7]], dtype=torch.int32, device=DEV)
    out, path = torch.empty(b, seq, heads, dim, dtype=torch.bfloat16, device=DEV), torch.empty(b, seq, dtype=torch.int32, device=DEV)
    accepted, nxt = torch.empty(b, dtype=torch.int32, device=DEV), torch.empty(b, dtype=torch.int32, device=DEV)
    ws, q_out = workspace(out, kv), torch.empty_like(out)

    def step():
        positions = c.len[:, None] + depths
        hf.cache_append(qkv[:, :, heads:heads + kv], qkv[:, :, heads + kv:], c.k, c.v, c.table, c.len, q=qkv[:, :, :heads], q_out=q_out,
                        positions=positions, turns=turns)
        hf.cache_attention(q_out, c.k, c.v, c.table, c.len, out, mask=mask, workspace=ws)
        hf.tree_accept(tokens, up, picks, path, accepted, nxt, k_cache=c.k, v_cache=c.v, pages=c.table, lengths=c.len)
        c.len += accepted

    saved = [t.clone() for t in (*c.stores, c.len)]

    def again():
        for t, s in zip((*c.stores, c.len), saved):
            t.copy_(s)

    runs = []
    for how in ("called", "captured", "captured"):
        again()
        if how == "captured":
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
            again()
            go = g.replay
        else:
            go = step
        seen = []
        for _ in range(4):
            go()
            torch.cuda.synchronize()
            seen.append([t.clone() for t in (out, path, accepted, nxt, c.len, q_out)])
        runs.append(seen + [[c.raw(s).view(torch.int16).clone() for s in c.stores]])
    assert runs[0][0][2].tolist() == [3, 3] and runs[0][0][1][0].tolist() == [0, 2, 3, -1, -1] and runs[0][0][4].tolist() == [33, 10]
    for other in runs[1:]:
        for x, y in zip(runs[0], other):
            assert all(torch.equal(a, b) for a, b in zip(x, y))


def test_on_another_stream_and_beside_another_call():
    rng = np.random.default_rng(41)
    c = ref.filled(rng, [3000, 500], [4, 4], 4, 2, 128, 16, "bf16", DEV)
    q = ref.normal(rng, (2, 4, 8, 128), "bf16").to(DEV)
    want = hf.cache_attention(q, c.k, c.v, c.table, c.len, torch.empty_like(q), workspace=workspace(q, 2))
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs, spaces = [torch.empty_like(q) for _ in streams], [workspace(q, 2) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, o, w in zip(streams, outs, spaces):
            with torch.cuda.stream(s):
                hf.cache_attention(q, c.k, c.v, c.table, c.len, o, workspace=w)
    torch.cuda.synchronize()
    assert all(torch.equal(want, o) for o in outs)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes: entries in its last pages."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough memory")
    kv, dim, page, pages = 8, 128, 64, 70000  # 4.6e9 elements each
    k, v = (torch.zeros(pages, page, kv, dim, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    rng = np.random.default_rng(42)
    for seq in (3, 40):
        n = 150
        ids = np.array([pages - 1, 2, pages - 3, 34000, 65536])[:-(-(n + seq) // page)]
        small = ref.filled(rng, [n], [0], seq, kv, dim, page, "bf16", DEV, spare=0)
        table = torch.from_numpy(ids.astype(np.int32)[None]).to(DEV)
        for a, s in ((k, small.k), (v, small.v)):
            a[ids[:small.width]] = torch.nan_to_num(s[small.table[0].long()])
        qkv = ref.normal(rng, (1, seq, 32 + 2 * kv, dim), "bf16").to(DEV)
        q, nk, nv = qkv[:, :, :32].contiguous(), qkv[:, :, 32:32 + kv], qkv[:, :, 32 + kv:]
        outs = []
        for kk, vv, t in ((k, v, table), (small.k, small.v, small.table)):
            hf.cache_append(nk, nv, kk, vv, t, small.len)
            outs.append(hf.cache_attention(q, kk, vv, t, small.len, torch.empty_like(q), workspace=workspace(q, kv)))
        assert torch.equal(*outs) and bool(torch.isfinite(outs[0]).all())


def test_versions_move():
    rng = np.random.default_rng(43)
    c = ref.filled(rng, [5], [1], 1, 1, 16, 16, "f32", DEV)
    q = ref.normal(rng, (1, 1, 2, 16), "f32").to(DEV)
    out, ws = torch.empty_like(q), workspace(q, 1)
    old = [t._version for t in (c.k, c.v, out, ws)]
    hf.cache_append(q[:, :, :1], q[:, :, :1], c.k, c.v, c.table, c.len)
    hf.cache_attention(q, c.k, c.v, c.table, c.len, out, workspace=ws)
    assert all(t._version > o for t, o in zip((c.k, c.v, out, ws), old))


def test_the_binding_refuses_other_tensors(monkeypatch):
    """With the launch switched off: nothing that should have been refused reaches the device."""
    monkeypatch.setenv("HLOFUSION_FAULT", "all")
    new = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device=DEV)  # noqa: E731
    i32 = torch.int32
    base = dict(q=new(2, 3, 4, 16), k=new(9, 4, 2, 16), v=new(9, 4, 2, 16), table=new(2, 5, t=i32), lengths=new(2, t=i32), out=new(2, 3, 4, 16),
                ws=new(1 << 24, t=torch.uint8))

    def attention(counts=None, mask=None, lse=None, **kw):
        a = {**base, **kw}
        return hf.cache_attention(a["q"], a["k"], a["v"], a["table"], a["lengths"], a["out"], counts=counts, mask=mask, lse=lse, workspace=a["ws"])

    def status(call):
        with pytest.raises(hf.HloError) as e:
            call()
        return e.value.status

    assert status(attention) == 3
    i64 = torch.int64
    for kw in (dict(lengths=new(2, t=i64)), dict(lengths=new(3, t=i32)), dict(lengths=None), dict(table=new(2, 5, t=i64)), dict(counts=new(2, t=i64)),
               dict(counts=new(4, t=i32)[::2]), dict(mask=new(2, 3, 1, t=i64)), dict(lse=new(2, 3, 3)), dict(lse=new(2, 3, 4, t=torch.float16)),
               dict(q=new(2, 3, 4, 16).cpu()), dict(k=new(9, 4, 2, 16, t=torch.float64)), dict(ws=new(1 << 24, t=torch.uint8).cpu()),
               dict(lengths=new(2, t=i32).cpu()), dict(k=None)):
        assert status(lambda: attention(**kw)) == 1, kw
    assert status(lambda: attention(ws=new(16, t=torch.uint8))) == 4
    q, k = base["q"], new(2, 3, 2, 16)
    append = lambda **kw: hf.cache_append(k, k, base["k"], base["v"], base["table"], base["lengths"], **kw)  # noqa: E731
    assert status(append) == 3 and status(lambda: append(q=q, q_out=base["out"], turns=new(8, t=i64))) == 3
    for kw in (dict(turns=new(8)), dict(turns=new(9, t=i64)), dict(turns=new(8, t=i64), n_pairs=9), dict(positions=new(2, 3, t=i64)), dict(q=q),
               dict(counts=new(3, t=i32))):
        assert status(lambda: append(**kw)) == 1, kw
    t = [new(2, 3, t=i32) for _ in range(4)]
    accept = lambda a, n, **kw: hf.tree_accept(*t, a, n, **kw)  # noqa: E731
    one, two = new(2, t=i32), new(2, t=i32)
    assert status(lambda: accept(one, two)) == 3
    assert status(lambda: accept(one, new(2, t=i64))) == 1 and status(lambda: accept(one, new(3, t=i32))) == 1
    assert status(lambda: accept(one, two, k_cache=base["k"])) == 1
