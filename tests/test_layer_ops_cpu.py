"""The fusions between a decoder's matrix products, without a GPU: the generator against its published
vectors, the rotary tables, and the refusals of every entry point (before anything touches the device)."""

import ctypes
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest

import layer_reference as ref
import transpose_heroes_gb300 as hf
from transpose_heroes_gb300 import build as hbuild

A, B, C, E, S = 0x10000000, 0x20000000, 0x30000000, 0x40000000, 0x50000000  # addresses never dereferenced
V = hf.DeviceView


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


# ---- the generator -----------------------------------------------------------------------------------------
@pytest.mark.parametrize("counter,key,words", [
    # the vectors published with the generator for Philox4x32-10
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_reference_generator_against_published_vectors(counter, key, words):
    got = ref.philox(key[0] | key[1] << 32, counter[2] | counter[3] << 32, [counter[0] | counter[1] << 32])
    assert tuple(int(w) for w in got[0]) == words


def test_reference_mask_keeps_its_share():
    for p in (0.0, 0.1, 0.5, 1.0):
        k = ref.keep(p, 7, 3, 1 << 16)
        assert abs(k.mean() - (1 - p)) <= 5 * math.sqrt(p * (1 - p) / (1 << 16))


# ---- rotary tables -----------------------------------------------------------------------------------------
def _theta(base, i, rot):
    return (Decimal(base).ln() * Decimal(-2 * i) / Decimal(rot)).exp()


PI = Decimal("3.14159265358979323846264338327950288419716939937510")


@pytest.mark.parametrize("rot", [2, 6, 64, 128])
@pytest.mark.parametrize("scaling,factor", [(None, 1), ("linear", 4), ("base", 8), ("by_parts", 8)])
def test_rotary_turns(rot, scaling, factor):
    """Against 50-digit arithmetic: theta in double precision (a power, a quotient) is within 2^-50 relative."""
    getcontext().prec = 50
    base, length, low, high = 10000, 8192, 1, 4
    if scaling == "base" and rot == 2:
        refused(lambda: hf.rotary_turns(rot, scaling="base", factor=2.0), word="two pairs")
        return
    got = hf.rotary_turns(rot, base, scaling, factor, length, low, high).view(np.uint64)
    for i in range(rot // 2):
        b = Decimal(base)
        if scaling == "base":
            b = b * (Decimal(factor).ln() * Decimal(rot) / Decimal(rot - 2)).exp()
        th = _theta(b, i, rot)
        if scaling == "linear":
            th /= factor
        if scaling == "by_parts":
            w = Decimal(length) * th / (2 * PI)
            g = min(Decimal(1), max(Decimal(0), (w - low) / Decimal(high - low)))
            th *= g + (1 - g) / factor
        want = th / (2 * PI) * Decimal(2) ** 64
        # the power's exponent is up to ln(base) long, so its rounding counts ten times over; the mixture
        # amplifies the error of g by (1 - 1 / factor) w / (high - low) <= 8 at most
        assert abs(Decimal(int(got[i])) - want) <= want * Decimal(2) ** -45 + 1, i


def test_rotary_turns_refusals():
    refused(lambda: hf.rotary_turns(7))
    refused(lambda: hf.rotary_turns(8, base=0.5), word="base")
    refused(lambda: hf.rotary_turns(8, base=math.inf), word="base")
    refused(lambda: hf.rotary_turns(8, scaling="linear", factor=0.5), word="factor")
    refused(lambda: hf.rotary_turns(8, scaling="by_parts", factor=2, original_length=0), word="by parts")
    refused(lambda: hf.rotary_turns(8, scaling="by_parts", factor=2, original_length=10, low=4, high=4), word="by parts")
    assert hf.rotary_turns(0).size == 0


# ---- views -------------------------------------------------------------------------------------------------
def test_view_refusals():
    x = V(A, [4, 8], "f32")
    refused(lambda: hf.rms_norm(V(A, [4, 8], "f32", [16, 2]), V(B, [4, 8], "f32"), stream=0), 2, "stride must be 1")
    refused(lambda: hf.rms_norm(V(A, [4, 8], "f32", [-8, 1]), V(B, [4, 8], "f32"), stream=0), word="negative stride")
    refused(lambda: hf.rms_norm(V(A, [4, -8], "f32", [8, 1]), V(B, [4, 8], "f32"), stream=0), word="negative size")
    refused(lambda: hf.rms_norm(x, V(B, [4, 8], "f32", [4, 1]), stream=0), word="output elements overlap")
    refused(lambda: hf.rms_norm(x, V(B, [4, 8], "f32", [0, 1]), stream=0), word="output elements overlap")
    refused(lambda: hf.rms_norm(x, V(B + 2, [4, 8], "f32"), stream=0), word="aligned")
    refused(lambda: hf.rms_norm(x, V(0, [4, 8], "f32"), stream=0), word="NULL")
    refused(lambda: hf.rms_norm(x, None, stream=0), word="NULL")
    refused(lambda: hf.rms_norm(V(A, [], "f32"), V(B, [], "f32"), stream=0), word="rank")
    refused(lambda: hf.rms_norm(V(A, [1 << 40, 1 << 30], "f32"), V(B, [1 << 40, 1 << 30], "f32"), stream=0), word="too large")
    refused(lambda: V(A, [1] * 9, "f32"), word="dimensions")
    refused(lambda: hf.rms_norm(V(A, [4, 8], "s32"), V(B, [4, 8], "s32"), stream=0), 2, "not supported")


def test_in_place_and_interleaved_views(monkeypatch):
    x, y = V(A, [4, 8], "bf16"), V(A, [4, 8], "bf16")
    accepted(lambda: hf.rms_norm(x, y, stream=0), monkeypatch)  # exactly in place
    monkeypatch.delenv("HLOFUSION_FAULT")
    refused(lambda: hf.rms_norm(x, V(A + 2, [4, 8], "bf16"), stream=0), word="overlaps")
    refused(lambda: hf.rms_norm(x, V(A, [4, 8], "f32"), stream=0), word="overlaps")  # another type
    refused(lambda: hf.rms_norm(x, V(A, [4, 8], "bf16", [16, 1]), stream=0), word="overlaps")  # other strides
    # sum and out on one buffer, even with one descriptor for both
    out = V(B, [4, 8], "bf16")
    refused(lambda: hf.rms_norm(x, out, residual=V(C, [4, 8], "bf16"), sum_out=out, stream=0), word="overlaps")
    # two halves of rows of 16: provably apart; shifted by one element: not
    accepted(lambda: hf.rms_norm(V(A, [4, 8], "bf16", [16, 1]), V(A + 16, [4, 8], "bf16", [16, 1]), stream=0), monkeypatch)
    monkeypatch.delenv("HLOFUSION_FAULT")
    refused(lambda: hf.rms_norm(V(A, [4, 8], "bf16", [16, 1]), V(A + 14, [4, 8], "bf16", [16, 1]), stream=0), word="overlaps")
    refused(lambda: hf.rms_norm(V(A, [4, 8], "bf16", [16, 1]), V(A + 18, [4, 8], "bf16", [16, 1]), stream=0), word="overlaps")
    # an operand broadcast over the rows
    accepted(lambda: hf.rms_norm(x, out, residual=V(C, [4, 8], "bf16", [0, 1]), stream=0), monkeypatch)


def test_rms_norm_refusals(monkeypatch):
    x, out = V(A, [4, 8], "bf16"), V(B, [4, 8], "bf16")
    s8, f8 = V(B, [4, 8], "s8"), V(B, [4, 8], "f8e4m3fn")
    refused(lambda: hf.rms_norm(x, V(B, [4, 9], "bf16"), stream=0), word="expected 8")
    refused(lambda: hf.rms_norm(x, V(B, [32], "bf16"), stream=0), word="rank")
    refused(lambda: hf.rms_norm(V(A, [4, 0], "bf16"), V(B, [4, 0], "bf16"), stream=0), word="empty")
    refused(lambda: hf.rms_norm(x, V(B, [4, 8], "f16"), stream=0), word="type")
    refused(lambda: hf.rms_norm(x, s8, stream=0), word="8 bits")
    refused(lambda: hf.rms_norm(x, f8, stream=0), word="8 bits")
    refused(lambda: hf.rms_norm(x, out, scales=S, stream=0), word="scales belong")
    q = {"host_scales": np.float32([0.1]), "host_zero_points": np.int32([0]), "quantization_dimension": None}
    refused(lambda: hf.rms_norm(x, s8, scales=S, out_q=q, stream=0), word="exclude")
    refused(lambda: hf.rms_norm(x, f8, out_q=q, stream=0), word="out_q belongs")
    refused(lambda: hf.rms_norm(x, s8, out_q={**q, "host_scales": np.float32([0.0])}, stream=0), word="C6")
    refused(lambda: hf.rms_norm(x, out, residual=V(C, [4, 8], "f32"), stream=0), word="differs")
    refused(lambda: hf.rms_norm(x, out, sum_out=V(C, [4, 8], "f32"), stream=0), word="differs")
    refused(lambda: hf.rms_norm(x, out, eps=-1.0, stream=0), word="eps")
    refused(lambda: hf.rms_norm(x, out, eps=math.nan, stream=0), word="eps")
    refused(lambda: hf.rms_norm(x, out, weight=C, weight_dtype="f16", stream=0), word="weight type")
    refused(lambda: hf.rms_norm(x, out, weight=B + 32, weight_dtype="bf16", stream=0), word="overlaps")
    refused(lambda: hf.rms_norm(x, out, rstd=S + 2, stream=0), word="aligned")
    refused(lambda: hf.rms_norm(x, out, rstd=B, stream=0), word="overlaps")
    refused(lambda: hf.rms_norm(x, s8, scales=S, rstd=S + 8, stream=0), word="overlaps")
    for p in (-0.1, 1.1, math.nan):
        refused(lambda: hf.rms_norm(x, out, dropout=hf.Dropout(p, 1, 2), stream=0), word="outside 0..1")
    refused(lambda: hf.rms_norm(x, out, dropout=hf.Dropout(0.5, 1, 2, state=S + 4), stream=0), word="8-byte")
    for o, kw in [(out, {}), (V(B, [4, 8], "f32"), {}), (s8, {"scales": S}), (f8, {"scales": S}), (s8, {"out_q": q})]:
        accepted(lambda: hf.rms_norm(x, o, stream=0, **kw), monkeypatch)
    monkeypatch.delenv("HLOFUSION_FAULT")
    hf.rms_norm(V(0, [0, 8], "f32"), V(0, [0, 8], "f32"), stream=0)  # no rows: nothing to do


def test_rms_norm_backward_refusals(monkeypatch):
    dy, h, dh, dx = (V(p, [4, 8], "f32") for p in (A, B, C, E))
    run = lambda **kw: hf.rms_norm_backward(**{**dict(dy=dy, h=h, rstd=S, dh=dh, stream=0), **kw})
    refused(lambda: run(dx=dx), word="dropout")
    refused(lambda: run(dropout=hf.Dropout(0.5)), word="dropout")
    refused(lambda: run(rstd=None), word="rstd is NULL")
    refused(lambda: run(dy=V(A, [4, 8], "bf16")), word="differs")
    refused(lambda: run(dsum=V(E, [4, 7], "f32")), word="expected 8")
    refused(lambda: run(dh=V(A + 4, [4, 8], "f32")), word="overlaps")
    refused(lambda: run(dx=dh, dropout=hf.Dropout(0.5)), word="overlaps")
    need = hf.rms_norm_workspace_size(4, 8)
    assert need >= 4 * 8
    refused(lambda: run(dweight=S + 4096), 4, "workspace")
    refused(lambda: run(dweight=S + 4096, workspace=S + 8192, workspace_bytes=need - 1), 4, "workspace")
    refused(lambda: run(dweight=S + 4096, workspace=S + 8196, workspace_bytes=need), word="16-byte")
    refused(lambda: run(dweight=S + 4096, workspace=A, workspace_bytes=need), word="overlaps")
    refused(lambda: run(dweight=S, workspace=S + 8192, workspace_bytes=need), word="overlaps")
    accepted(lambda: run(dweight=S + 4096, workspace=S + 8192, workspace_bytes=need), monkeypatch)
    accepted(lambda: run(dh=V(A, [4, 8], "f32")), monkeypatch)
    assert hf.rms_norm_workspace_size(0, 8) == 0 and hf.rms_norm_workspace_size(8, 0) == 0


def test_dropout_refusals(monkeypatch):
    x, out, d = V(A, [4, 8], "f16"), V(B, [4, 8], "f16"), hf.Dropout(0.5, 1, 2)
    refused(lambda: hf.dropout(x, out, None, stream=0), word="NULL")
    refused(lambda: hf.dropout(x, V(B, [4, 8], "f32"), d, stream=0), word="one element type")
    refused(lambda: hf.dropout(x, out, d, residual=V(C, [4, 8], "f32"), stream=0), word="one element type")
    refused(lambda: hf.dropout(x, out, d, residual=V(C, [8, 4], "f16"), stream=0), word="expected")
    refused(lambda: hf.dropout(x, V(A + 4, [4, 8], "f16"), d, stream=0), word="overlaps")
    refused(lambda: hf.dropout(x, out, hf.Dropout(2.0), stream=0), word="outside")
    refused(lambda: hf.dropout(V(A, [4], "s8"), V(B, [4], "s8"), d, stream=0), 2)
    accepted(lambda: hf.dropout(x, x, d, stream=0), monkeypatch)


def test_rotary_refusals(monkeypatch):
    x, out, pos = V(A, [2, 3, 4, 16], "bf16"), V(B, [2, 3, 4, 16], "bf16"), V(S, [2, 3], "s32")
    run = lambda **kw: hf.rotary(**{**dict(x=x, out=out, positions=pos, turns=C, n_pairs=8, stream=0), **kw})
    refused(lambda: run(x=V(A, [3, 16], "bf16")), word="rank")
    refused(lambda: run(n_pairs=9), word="pairs")
    refused(lambda: run(n_pairs=-1), word="pairs")
    refused(lambda: run(turns=0), word="turns is NULL")
    refused(lambda: run(turns=C + 4), word="8-byte")
    refused(lambda: run(positions=V(S, [3, 2], "s32")), word="positions")
    refused(lambda: run(positions=V(S, [6], "s32")), word="positions")
    refused(lambda: run(positions=V(S, [2, 3], "f32")), word="s32")
    refused(lambda: run(scale=math.inf), word="scale")
    refused(lambda: run(out=V(B, [2, 3, 4, 16], "f32")), word="one element type")
    refused(lambda: run(k=V(E, [2, 3, 1, 16], "bf16")), word="together")
    refused(lambda: run(k=V(E, [2, 3, 1, 8], "bf16"), k_out=V(E + 4096, [2, 3, 1, 8], "bf16")), word="rotary y")
    refused(lambda: run(out=V(A + 32, [2, 3, 4, 16], "bf16")), word="overlaps")
    refused(lambda: run(k=V(E, [2, 3, 1, 16], "bf16"), k_out=V(B, [2, 3, 1, 16], "bf16")), word="overlaps")
    # queries and keys of a packed projection, each in place; but not one onto the other
    q = V(A, [2, 3, 4, 16], "bf16", [288, 96, 16, 1])
    k = V(A + 128, [2, 3, 1, 16], "bf16", [288, 96, 16, 1])
    accepted(lambda: run(x=q, out=q, k=k, k_out=k), monkeypatch)
    monkeypatch.delenv("HLOFUSION_FAULT")
    refused(lambda: run(x=q, out=q, k=V(E, [2, 3, 1, 16], "bf16"), k_out=V(A + 96, [2, 3, 1, 16], "bf16", [288, 96, 16, 1])),
            word="overlaps")
    # packed projections of sequences with a gap between them
    q = V(A, [2, 3, 4, 16], "bf16", [1000, 96, 16, 1])
    k = V(A + 128, [2, 3, 1, 16], "bf16", [1000, 96, 16, 1])
    accepted(lambda: run(x=q, out=q, k=k, k_out=k), monkeypatch)


def test_logits_refusals(monkeypatch):
    x, out, hist = V(A, [3, 70], "bf16"), V(B, [3, 70], "bf16"), V(C, [3, 5], "s32")
    run = lambda **kw: hf.logits_process(**{**dict(logits=x, out=out, stream=0), **kw})
    refused(lambda: run(out=None), word="neither")
    refused(lambda: run(logits=V(A, [3, 7, 10], "bf16")), word="rank")
    refused(lambda: run(logits=V(A, [3, 70], "s8")), 2)
    refused(lambda: run(out=V(B, [3, 70], "f16")), word="out")
    refused(lambda: run(bias=V(E, [3, 69], "f32")), word="bias")
    refused(lambda: run(bias=V(E, [3, 70], "bf16")), word="f32")
    refused(lambda: run(history=V(C, [2, 5], "s32")), word="history")
    refused(lambda: run(mask=V(E, [3, 2], "s32")), word="mask")
    refused(lambda: run(lengths=S), word="history")
    refused(lambda: run(repetition=S), word="history")
    refused(lambda: run(history=hist, lengths=S + 2), word="aligned")
    refused(lambda: run(history=hist, lengths=S, token=S + 4), word="overlaps")
    refused(lambda: run(token=A), word="overlaps")
    refused(lambda: run(out=V(A + 2, [3, 70], "bf16")), word="overlaps")
    refused(lambda: run(out=V(C, [3, 70], "bf16"), history=hist), word="overlaps")
    accepted(lambda: run(out=x, history=hist, mask=V(E, [3, 3], "s32"), token=S), monkeypatch)
    accepted(lambda: run(out=V(B, [3, 70], "f32"), bias=V(E, [3, 70], "f32", [0, 1])), monkeypatch)


def test_tensors_must_be_on_the_gpu():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8)
    refused(lambda: hf.rms_norm(x, V(B, [4, 8], "f32"), stream=0), word="on the GPU")
    refused(lambda: hf.rms_norm(V(A, [4, 8], "f32"), V(B, [4, 8], "f32"), weight=torch.ones(8), stream=0), word="on the GPU")
    refused(lambda: hf.rms_norm(x.to_sparse(), V(B, [4, 8], "f32"), stream=0))
    with pytest.raises(TypeError):
        hf.rms_norm(3, V(B, [4, 8], "f32"), stream=0)


def test_a_dropout_state_is_two_64_bit_words_on_the_gpu():
    torch = pytest.importorskip("torch")
    for state in (torch.zeros(2), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int64), torch.zeros(3, dtype=torch.int64),
                  torch.zeros(4, dtype=torch.int64)[::2]):
        refused(lambda: hf.Dropout(0.5, 1, 2, state), word="64-bit")
    refused(lambda: hf.Dropout(0.5, 1, 2, torch.zeros(2, dtype=torch.int64)), word="on the GPU")
    assert hf.Dropout(0.5, 1, 2, S).state == S


def test_parameters_are_of_their_own_type():
    """Not any buffer of the same size."""
    x, y = V(A, [4, 8], "f32"), V(B, [4, 8], "f32")
    for d in (np.zeros(4), bytes(32), 0.5, (ctypes.c_double * 4)()):
        with pytest.raises(TypeError):
            hf.dropout(x, y, d, stream=0)
        with pytest.raises(TypeError):
            hf.rms_norm(x, y, dropout=d, stream=0)


def test_a_views_tensor_must_be_on_the_gpu():
    torch = pytest.importorskip("torch")
    refused(lambda: V(torch.zeros(4, 8), [4, 8], "f32"), word="on the GPU")
    assert V(A, [4, 8], "f32").ptr == A and V(None, [0, 8], "f32").ptr == 0


def test_the_library_builds_without_torch(monkeypatch, tmp_path):
    """nvcc is enough for it; the extension is left out."""
    import sys

    monkeypatch.setitem(sys.modules, "torch", None)  # as if it were not installed
    monkeypatch.setattr(hbuild, "CALL", str(tmp_path / "_hlocall.so"))
    assert hbuild.build() == hbuild.LIB
    assert not list(tmp_path.iterdir())


def test_an_extension_of_another_torch_is_not_loaded(monkeypatch, tmp_path):
    """... and is not up to date."""
    pytest.importorskip("torch")
    import shutil

    call = str(tmp_path / "_hlocall.so")
    shutil.copy(hbuild.CALL, call)
    (tmp_path / "_hlocall.so.abi").write_text("torch 1.0, another")
    monkeypatch.setattr(hf, "CALL_PATH", call)
    monkeypatch.setattr(hf, "_call", None)
    with pytest.raises(RuntimeError, match="built for torch 1.0"):
        hf.dropout(V(A, [4], "f32"), V(B, [4], "f32"), hf.Dropout(0.5), stream=0)
    assert hbuild.built_for(call) != hbuild.call_abi() == hbuild.built_for()


def test_side_outputs_over_the_generators_state(monkeypatch):
    x, y, s8, h = V(A, [4, 8], "f32"), V(B, [4, 8], "f32"), V(B, [4, 8], "s8"), V(C, [4, 8], "f32")
    at = lambda p: hf.Dropout(0.5, 1, 2, state=p)  # noqa: E731
    refused(lambda: hf.rms_norm(x, y, rstd=S, dropout=at(S + 8), stream=0), word="state")
    refused(lambda: hf.rms_norm(x, s8, scales=S + 8, dropout=at(S), stream=0), word="state")
    need = hf.rms_norm_workspace_size(4, 8)
    run = lambda d, w, p: hf.rms_norm_backward(x, h, S, y, dx=V(E, [4, 8], "f32"), dropout=at(p), dweight=d, workspace=w,  # noqa: E731
                                               workspace_bytes=need, stream=0)
    refused(lambda: run(S + 4096, S + 8192, S + 4096 + 24), word="state")
    refused(lambda: run(S + 4096, S + 8192, S + 8192), word="state")
    accepted(lambda: run(S + 4096, S + 8192, S + 16), monkeypatch)
    accepted(lambda: hf.rms_norm(x, y, rstd=S, dropout=at(S + 16), stream=0), monkeypatch)


def test_f8_is_no_type_of_the_other_entry_points():
    a = hf.make_array([4, 5], None, "f32")
    a.dtype = 5
    o = hf.make_array([4], None, "f32")
    dims = (ctypes.c_int64 * 1)(1)
    st = hf.lib().hlo_reduce_fusion(ctypes.byref(a), A, None, dims, 1, 0, 0.0, 0, ctypes.byref(o), B, None, 0, 0)
    assert st == 1 and "unknown element type" in hf.last_error()
