"""The paged cache's operators without a GPU: the tree's mask, and the refusals of every entry point (before anything touches
the device)."""

import numpy as np
import pytest

import transpose_heroes_gb300 as hf
from transpose_heroes_gb300 import build as hbuild

V = hf.DeviceView
K, VV, T, L, Q, O, W, M, S, X = (0x10000000 * (i + 1) for i in range(10))  # addresses never dereferenced
MB = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def lib():
    hbuild.build()
    return hf.lib()


def refused(call, status=1, word=""):
    with pytest.raises(hf.HloError) as e:
        call()
    assert e.value.status == status and word in str(e.value), str(e.value)


def accepted(call, monkeypatch):
    """Passes validation: the injected fault answers in place of the launch."""
    monkeypatch.setenv("HLOFUSION_FAULT", "all")
    with pytest.raises(hf.HloError) as e:
        call()
    assert e.value.status == 3 and "injected fault" in str(e.value), str(e.value)
    monkeypatch.delenv("HLOFUSION_FAULT")


# ---- the tree's mask -------------------------------------------------------------------------------------------
@pytest.mark.parametrize("n", [0, 1, 2, 31, 32, 33, 100, 1000])
def test_tree_mask(n):
    rng = np.random.default_rng(n)
    parents = [int(rng.integers(-1, c)) if c else -1 for c in range(n)]
    mask, depths = hf.tree_mask(parents)
    assert mask.shape == (n, (n + 31) // 32) and mask.dtype == depths.dtype == np.int32
    bits = mask.view(np.uint32)
    for c in range(n):
        seen, u = set(), c
        while u >= 0:
            seen.add(u)
            u = parents[u]
        got = {32 * w + k for w in range(bits.shape[1]) for k in range(32) if bits[c, w] >> k & 1}
        assert got == seen and depths[c] == len(seen) - 1


def test_tree_mask_refuses():
    refused(lambda: hf.tree_mask([-1, 1]), word="parent of node 1")
    refused(lambda: hf.tree_mask([-1, -2]), word="parent of node 1")
    refused(lambda: hf.tree_mask([0]), word="parent of node 0")
    refused(lambda: hf.tree_mask([[-1]]), word="rank 2")


# ---- attention -------------------------------------------------------------------------------------------------
def attention(q=(2, 3, 8, 64), cache=(20, 16, 2, 64), v=None, table=(2, 5), out=None, dtype="bf16", cdtype=None, vdtype=None, tdtype="s32",
              odtype=None, mask=None, mdtype="s32", qp=Q, kp=K, vp=VV, tp=T, op=O, lp=L, wp=W, mp=M, bytes_=1 << 30, kstr=None, qstr=None, ostr=None,
              **kw):
    cdtype = cdtype or dtype
    return hf.cache_attention(V(qp, q, dtype, qstr), V(kp, cache, cdtype, kstr), V(vp, v or cache, vdtype or cdtype), V(tp, table, tdtype), lp,
                              V(op, out or q, odtype or dtype, ostr), mask=None if mask is None else V(mp, mask, mdtype), workspace=wp,
                              workspace_bytes=bytes_, stream=S, **kw)


def test_attention_takes(monkeypatch):
    for call in (lambda: attention(), lambda: attention(mask=(2, 3, 1)), lambda: attention(mask=(3, 1)), lambda: attention(lse=X, counts=X + MB),
                 lambda: attention(cdtype="f8e4m3fn", k_scale=0.1, v_scale=3.0), lambda: attention(dtype="f32"), lambda: attention(op=Q),
                 lambda: attention(cache=(20, 16, 8, 64)), lambda: attention(table=(2, 0)), lambda: attention(q=(2, 3, 8, 256), cache=(20, 1, 1, 256)),
                 lambda: attention(vp=K), lambda: attention(scale=2.0)):
        accepted(call, monkeypatch)
    need = hf.cache_attention_workspace_size(2, 3, 8, 2, 64)
    accepted(lambda: attention(bytes_=need), monkeypatch)
    refused(lambda: attention(bytes_=need - 1), 4, "workspace of")


def test_attention_of_nothing():
    """No launch."""
    assert attention(q=(0, 3, 8, 64), table=(0, 5), lp=None, wp=None, bytes_=0) is not None
    assert attention(q=(2, 0, 8, 64), wp=None, bytes_=0) is not None
    assert attention(q=(2, 3, 0, 64), wp=None, bytes_=0) is not None
    for shape in ((0, 1, 8, 2, 64), (1, 0, 8, 2, 64), (1, 1, 8, 2, 257), (1, 1, 0, 2, 64), (1, 1, 8, -1, 64)):
        assert hf.cache_attention_workspace_size(*shape) == 0


def test_attention_refuses():
    refused(lambda: attention(q=(2, 3, 64)), word="rank")
    refused(lambda: attention(cache=(16, 2, 64)), word="rank")
    refused(lambda: attention(cache=(3, 20, 16, 2, 64)), word="rank")
    refused(lambda: attention(table=(2, 5, 1)), word="rank")
    refused(lambda: attention(table=(3, 5)), word="sequences")
    refused(lambda: attention(tdtype="f32"), word="s32")
    refused(lambda: attention(cache=(20, 16, 3, 64)), word="multiple")
    refused(lambda: attention(cache=(20, 16, 0, 64)), word="multiple")
    refused(lambda: attention(cache=(20, 0, 2, 64)), word="no entries")
    refused(lambda: attention(cache=(20, 16, 2, 32)), word="elements")
    refused(lambda: attention(v=(20, 16, 2, 32)), word="v_cache")
    refused(lambda: attention(vdtype="f16"), word="v_cache")
    refused(lambda: attention(cdtype="f16"), word="type")
    refused(lambda: attention(odtype="f32"), word="type")
    refused(lambda: attention(out=(2, 3, 8, 32)), word="dimension")
    refused(lambda: attention(dtype="s8"), 2, "element type")
    refused(lambda: attention(q=(2, 3, 8, 257), cache=(20, 16, 2, 257)), 2, "1 to 256")
    refused(lambda: attention(q=(2, 3, 8, 0), cache=(20, 16, 2, 0)), 2, "1 to 256")
    refused(lambda: attention(k_scale=0.5), word="f8E4M3FN")
    for bad in (0.0, -1.0, float("nan"), float("inf"), 1e-60, 1e60):
        refused(lambda: attention(cdtype="f8e4m3fn", v_scale=bad), word="finite")
        refused(lambda: attention(scale=bad), word="scale")
    refused(lambda: attention(mask=(2, 3, 2)), word="mask")
    refused(lambda: attention(mask=(2, 4, 1)), word="mask")
    refused(lambda: attention(mask=(2, 3, 1), mdtype="f32"), word="mask")
    refused(lambda: attention(lp=None), word="lengths")
    refused(lambda: attention(lp=L + 2), word="aligned")
    refused(lambda: attention(lse=X + 2), word="aligned")
    refused(lambda: attention(counts=X + 2), word="aligned")
    refused(lambda: attention(wp=W + 8), word="aligned")
    refused(lambda: attention(wp=None), 4, "workspace")
    refused(lambda: attention(table=(2, 1 << 27)), 2, "2^31")
    refused(lambda: attention(q=(1 << 20, 1 << 10, 8, 64), table=(1 << 20, 5)), 2, "new tokens")
    refused(lambda: attention(ostr=[0, 512, 64, 1]), word="overlap")
    refused(lambda: attention(qstr=[1536, 512, 64, 2]), 2, "stride")
    refused(lambda: hf.cache_attention(V(Q, (2, 3, 8, 64), "bf16"), None, None, None, None, V(O, (2, 3, 8, 64), "bf16"), workspace=W, workspace_bytes=1, stream=S), word="wanted")


def test_attention_refuses_overlaps():
    refused(lambda: attention(op=Q + 128), word="overlaps")
    refused(lambda: attention(op=K + 128), word="overlaps")
    refused(lambda: attention(op=T - 128), word="overlaps")
    refused(lambda: attention(op=L - 128), word="overlaps")
    refused(lambda: attention(mask=(2, 3, 1), mp=O + 4), word="overlaps")
    for place in (Q, K, VV, T, L, O, W):
        refused(lambda: attention(lse=place), word="overlaps")
    for place in (Q, K, VV, T, L, O):
        refused(lambda: attention(wp=place), word="overlaps")
    refused(lambda: attention(counts=X, lse=X), word="overlaps")


# ---- appending ---------------------------------------------------------------------------------------------------
def append(k=(2, 3, 2, 64), v=None, cache=(20, 16, 2, 64), table=(2, 5), q=(2, 3, 8, 64), qo=None, dtype="bf16", cdtype=None, qdtype=None, kp=Q,
           vp=Q + MB, ckp=K, cvp=VV, tp=T, lp=L, qp=Q + 2 * MB, op=O, positions=None, pdtype="s32", turns=X, n_pairs=32, cstr=None, cvstr=None, **kw):
    return hf.cache_append(V(kp, k, dtype), V(vp, v or k, dtype), V(ckp, cache, cdtype or dtype, cstr), V(cvp, cache, cdtype or dtype, cvstr),
                           V(tp, table, "s32"), lp, q=None if q is None else V(qp, q, qdtype or dtype), q_out=None if qo == 0 else V(op, qo or q, qdtype or dtype),
                           positions=None if positions is None else V(M, positions, pdtype), turns=turns, n_pairs=n_pairs, stream=S, **kw)


def test_append_takes(monkeypatch):
    inter = [2 * 16 * 2 * 64, 2 * 64, 64, 1]
    for call in (lambda: append(), lambda: append(q=None, qo=0), lambda: append(positions=(2, 3)), lambda: append(turns=None, n_pairs=None),
                 lambda: append(cdtype="f8e4m3fn", k_scale=0.1, v_scale=2.0), lambda: append(op=Q + 2 * MB), lambda: append(counts=M),
                 lambda: append(table=(2, 0)), lambda: append(dtype="f32"),
                 # keys and values of a page side by side in one buffer
                 lambda: append(cstr=inter, cvstr=inter, cvp=K + 16 * 2 * 64 * 2)):
        accepted(call, monkeypatch)


def test_append_refuses():
    refused(lambda: append(k=(2, 3, 64)), word="rank")
    refused(lambda: append(v=(2, 3, 2, 32)), word="v")
    refused(lambda: append(qo=0), word="go together")
    refused(lambda: append(q=(2, 4, 8, 64)), word="shape")
    refused(lambda: append(q=(2, 3, 8, 32)), word="shape")
    refused(lambda: append(qo=(2, 3, 4, 64)), word="q_out")
    refused(lambda: append(qdtype="f16"), word="element type")
    refused(lambda: append(cdtype="f16"), word="type")
    refused(lambda: append(dtype="s8"), 2, "element type")
    refused(lambda: append(cache=(20, 16, 4, 64)), word="heads")
    refused(lambda: append(cache=(20, 16, 2, 32)), word="heads")
    refused(lambda: append(table=(3, 5)), word="sequences")
    refused(lambda: append(k=(2, 3, 2, 513), cache=(20, 16, 2, 513), q=None, qo=0), 2, "512")
    refused(lambda: append(positions=(2, 4)), word="positions")
    refused(lambda: append(positions=(2, 3), pdtype="f32"), word="positions")
    refused(lambda: append(n_pairs=33), word="pairs")
    refused(lambda: append(n_pairs=-1), word="pairs")
    refused(lambda: append(turns=None, n_pairs=2), word="turns")
    refused(lambda: append(turns=X + 4), word="aligned")
    refused(lambda: append(counts=M + 1), word="aligned")
    refused(lambda: append(scale=float("nan")), word="scale")
    refused(lambda: append(k_scale=2.0), word="f8E4M3FN")
    refused(lambda: append(cstr=[2048, 0, 64, 1]), word="overlap")


def test_append_refuses_overlaps():
    refused(lambda: append(cvp=K), word="overlaps")
    refused(lambda: append(cvp=K + 4096), word="overlaps")
    for place in (Q, Q + MB, Q + 2 * MB, T, L, X):
        refused(lambda: append(ckp=place), word="overlaps")
    for place in (Q, Q + MB, Q + 2 * MB + 2, K, VV, T, L, X):
        refused(lambda: append(op=place), word="overlaps")
    refused(lambda: append(positions=(2, 3), op=M), word="overlaps")
    refused(lambda: append(counts=O), word="overlaps")


# ---- acceptance ----------------------------------------------------------------------------------------------------
def accept(shape=(2, 6), parents=None, picks=None, path=None, dtype="s32", tp=Q, pp=Q + MB, kp=Q + 2 * MB, op=O, ap=X, np_=X + MB, cache=None, table=(2, 5),
           ckp=K, cvp=VV, tb=T, lp=L, cdtype="bf16", **kw):
    with_ = {} if cache is None else dict(k_cache=V(ckp, cache, cdtype), v_cache=V(cvp, cache, cdtype), pages=V(tb, table, "s32"), lengths=lp)
    return hf.tree_accept(V(tp, shape, dtype), V(pp, parents or shape, "s32"), V(kp, picks or shape, "s32"), V(op, path or shape, "s32"), ap, np_, stream=S, **with_, **kw)


def test_accept_takes(monkeypatch):
    for call in (lambda: accept(), lambda: accept(parents=(6,)), lambda: accept(cache=(20, 16, 2, 64)), lambda: accept(cache=(7, 20, 16, 2, 64)),
                 lambda: accept(cache=(20, 16, 2, 64), cdtype="f8e4m3fn"), lambda: accept(counts=M), lambda: accept(shape=(2, 0)),
                 lambda: accept(shape=(1, 4096)), lambda: accept(cache=(20, 16, 0, 64))):
        accepted(call, monkeypatch)
    assert accept(shape=(0, 6), ap=None, np_=None) is not None


def test_accept_refuses():
    refused(lambda: accept(shape=(6,)), word="rank")
    refused(lambda: accept(dtype="f32"), word="s32")
    refused(lambda: accept(parents=(2, 5)), word="parents")
    refused(lambda: accept(picks=(3, 6)), word="picks")
    refused(lambda: accept(path=(2, 7)), word="path")
    refused(lambda: accept(shape=(1, 4097)), 2, "4096")
    refused(lambda: accept(ap=None), word="NULL")
    refused(lambda: accept(np_=X + MB + 2), word="aligned")
    refused(lambda: accept(cache=(2, 7, 20, 16, 2, 64)), word="rank")
    refused(lambda: accept(cache=(20, 16, 2, 64), table=(3, 5)), word="sequences")
    refused(lambda: accept(cache=(20, 16, 2, 64), lp=None), word="lengths")
    refused(lambda: accept(cache=(20, 16, 2, 64), cdtype="s8"), 2, "element type")


def test_accept_refuses_overlaps():
    for place in (Q, Q + MB, Q + 2 * MB):
        refused(lambda: accept(op=place), word="overlaps")
        refused(lambda: accept(ap=place), word="overlaps")
        refused(lambda: accept(np_=place), word="overlaps")
        refused(lambda: accept(cache=(20, 16, 2, 64), ckp=place), word="overlaps")
    refused(lambda: accept(ap=X, np_=X), word="overlaps")
    refused(lambda: accept(ap=O), word="overlaps")
    refused(lambda: accept(counts=X), word="overlaps")
    for place in (K, VV, T, L):
        refused(lambda: accept(cache=(20, 16, 2, 64), ap=place), word="overlaps")
        refused(lambda: accept(cache=(20, 16, 2, 64), op=place), word="overlaps")
    refused(lambda: accept(cache=(20, 16, 2, 64), cvp=K), word="overlaps")
