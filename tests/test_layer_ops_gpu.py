"""The fusions between a decoder's matrix products on the GPU against their plain 64-bit statements
(layer_reference.py). Bounds: the f32 error that reference derives for any order of summation, plus half a
unit of the output's type; masks, logits and greedy tokens are exact."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import layer_reference as ref
import transpose_heroes_gb300 as hf

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TYPES = ["f32", "bf16", "f16"]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transpose_heroes_gb300 import build

    build.build()
    hf.lib()


class Band:
    """A strided output inside a buffer filled with a pattern; check() wants every other byte untouched."""

    def __init__(self, dims, dtype, pitch=0, shift=0, heads_major=False):
        self.es = torch.empty(0, dtype=dtype).element_size()
        dims = list(dims)
        strides, s = [0] * len(dims), 1
        for i in range(len(dims) - 1, -1, -1):
            strides[i] = s
            s *= dims[i] + (pitch if i == len(dims) - 1 else 0)
        n = s + shift + 256
        self.raw = torch.full((n * self.es,), 0x5A, dtype=torch.uint8, device="cuda")
        self.t = self.raw.view(dtype).as_strided(dims, strides, 128 + shift)
        mask = torch.zeros(n, dtype=torch.bool, device="cuda")
        mask.as_strided(dims, strides, 128 + shift).fill_(True)
        self.outside = ~mask.repeat_interleave(self.es)

    def check(self):
        assert bool((self.raw[self.outside] == 0x5A).all()), "bytes outside the output were written"


def rnd(seed, *shape, std=1.0):
    return np.random.default_rng(seed).standard_normal(shape) * std


def dev(a, dtype, pitch=0, shift=0):
    """(device tensor of the rounded values, with a pitch and an odd start; those values in float64)."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DT.get(dtype, dtype))
    if pitch or shift:
        b = Band(t.shape, t.dtype, pitch, shift)
        b.t.copy_(t)
        return b.t, t.double().numpy()
    return t.cuda(), t.double().numpy()


def host(t):
    return t.detach().cpu().double().numpy()


def close(got, want, err, dtype, what=""):
    """|got - want| <= f32 error + half a unit of dtype (of the value, or of the subnormals)."""
    bound = err + (np.abs(want) + err) * ref.HALF_ULP[dtype] + ref.TINY[dtype]
    bad = ~(np.abs(host(got) - want) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.nanmax(np.abs(host(got) - want) / bound)} of the bound"


# n: one element, below a warp, ragged against every vector width, whole vectors, past a block's registers
SHAPES = [(1, 1), (3, 2), (2, 7), (5, 31), (37, 64), (3, 100), (9, 513), (2, 1000), (5, 1001), (3, 1024), (1, 4096), (7, 4104),
          (2, 5120), (1, 8191), (3, 8192), (2, 16385), (2, 33000), (1, 40000), (700, 72), (401, 129)]


def check_norm(rows, n, dtype, residual=True, weight="x", p=0.0, out="x", pitch=0, shift=0, w_offset=0.0, in_place=False,
               seed=0, state=False, eps=1e-6, std=1.0):
    x, xd = dev(rnd(seed + 1, rows, n, std=std), dtype, pitch, shift)
    r, rd = dev(rnd(seed + 2, rows, n, std=2 * std), dtype, pitch, shift) if residual else (None, None)
    w, wd = dev(1 + rnd(seed + 3, n, std=0.1), dtype if weight == "x" else "f32") if weight else (None, np.ones(n))
    d = (p, 0x123456789ABC + seed, 77) if p else None
    drop = None
    if d:
        st = torch.tensor([d[1], 70], dtype=torch.int64, device="cuda") if state else None
        drop = hf.Dropout(p, 5 if state else d[1], 7 if state else d[2], st)
    h, rs, y, eh, er, ey = ref.rms_norm(xd, wd, rd, w_offset, eps, d)
    rstd = torch.full((rows,), float("nan"), device="cuda")
    odt = {"x": DT[dtype], "f32": torch.float32, "s8": torch.int8, "static": torch.int8, "f8": torch.float8_e4m3fn}[out]
    ob = Band((rows, n), odt, pitch, shift)
    sb = Band((rows, n), DT[dtype], pitch, shift)
    if in_place:
        sb.t = r if residual else x
        sb.check = lambda: None
    scales = torch.full((rows,), float("nan"), device="cuda") if out in ("s8", "f8") else None
    q = {"host_scales": np.float32([0.05]), "host_zero_points": np.int32([3]), "quantization_dimension": None} if out == "static" else None
    hf.rms_norm(x, ob.t, weight=w, residual=r, sum_out=sb.t, rstd=rstd, eps=eps, weight_offset=w_offset, dropout=drop,
                scales=scales, out_q=q)
    torch.cuda.synchronize()
    ob.check(), sb.check()
    what = f"{rows}x{n} {dtype}"
    close(sb.t, h, eh, dtype, what + " sum")
    assert np.all(np.abs(host(rstd) - rs) <= rs * (er + 2 * ref.U) + 1e-45), what + " rstd"
    if out in ("x", "f32"):
        close(ob.t, y, ey, dtype if out == "x" else "f32", what + " out")
    elif out == "static":
        got = host(ob.t)
        t = y / np.float64(np.float32(0.05))
        lo, hi = (np.rint(t + s * (ey / 0.05 + np.abs(t) * 4 * ref.U)) for s in (-1, 1))
        assert np.all((got >= np.clip(lo + 3, -128, 127)) & (got <= np.clip(hi + 3, -128, 127))), what
    else:
        top = 127.0 if out == "s8" else 448.0
        want = np.abs(y).max(1) / top
        want[want < 2.0 ** -149 / 2] = 1.0
        es = (ey.max(1) / top + 4 * ref.U * want)
        s = host(scales)
        assert np.all(np.abs(s - want) <= es), what + " scales"
        t = y / s[:, None]
        et = ey / s[:, None] + np.abs(t) * 4 * ref.U
        got = host(ob.t.float())
        if out == "s8":
            assert np.all((got >= np.clip(np.rint(t - et), -128, 127)) & (got <= np.clip(np.rint(t + et), -128, 127))), what
        else:  # 3 bits of fraction: half a unit is 2^-4 relative, or 2^-10 among the subnormals
            assert np.all(np.abs(got - t) <= np.maximum(np.abs(t) * 2.0 ** -4, 2.0 ** -10) + et), what


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,n", SHAPES)
def test_rms_norm(rows, n, dtype):
    check_norm(rows, n, dtype)
    check_norm(rows, n, dtype, residual=False, weight="f32", p=0.3, seed=9)


@pytest.mark.parametrize("rows,n", [(310, 256), (310, 512), (320, 1000), (310, 1001), (310, 5120), (306, 8199)])
def test_rms_norm_of_many_rows(rows, n):
    """Past two rows an SM, where a thread holds several vectors."""
    check_norm(rows, n, "bf16", p=0.1)
    check_norm(rows, n, "f32", out="f32")


@pytest.mark.parametrize("out", ["x", "f32", "s8", "f8", "static"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,n", [(1, 1), (4, 8), (3, 77), (33, 256), (5, 1001), (2, 5120), (2, 8192), (1, 33001)])
def test_rms_norm_outputs(rows, n, dtype, out):
    check_norm(rows, n, dtype, out=out, w_offset=1.0, seed=20)
    check_norm(rows, n, dtype, out=out, weight=None, p=0.5, seed=30, state=True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pitch,shift", [(8, 0), (3, 0), (0, 1), (5, 3), (64, 8)])
@pytest.mark.parametrize("rows,n", [(7, 96), (5, 1001), (3, 4096)])
def test_rms_norm_strides(rows, n, pitch, shift, dtype):
    check_norm(rows, n, dtype, pitch=pitch, shift=shift, p=0.2)
    check_norm(rows, n, dtype, pitch=pitch, shift=shift, in_place=True, out="f8")


def test_rms_norm_mixed_strides_and_ranks():
    x, xd = dev(rnd(1, 3, 5, 40), "bf16")
    big = torch.zeros(5, 3, 2, 40, dtype=torch.bfloat16, device="cuda")
    out = big[:, :, 1].transpose(0, 1)  # [3, 5, 40], dimensions in another order, with gaps
    r, rd = dev(rnd(2, 5, 40), "bf16")  # one residual for every first index
    w, wd = dev(1 + rnd(3, 40), "bf16")
    hf.rms_norm(x, out, weight=w, residual=r.expand(3, 5, 40))
    _, _, y, _, _, ey = ref.rms_norm(xd, wd, np.broadcast_to(rd, xd.shape))
    close(out, y, ey, "bf16")
    assert bool((big[:, :, 0] == 0).all())


def test_rms_norm_long_rows_of_32_bits_in_place():
    check_norm(1, 70001, "f32", in_place=True, p=0.1)


@pytest.mark.parametrize("n", [40, 1001, 4096])
@pytest.mark.parametrize("out", ["x", "s8", "f8"])
def test_rms_norm_special_rows(n, out):
    """Zero rows, tiny rows, NaN and infinities stay in their rows."""
    x = torch.from_numpy(rnd(3, 6, n)).to(torch.bfloat16).cuda()
    x[0] = 0
    x[1, n // 2] = float("nan")
    x[2, 3] = float("inf")
    x[3] = 1e-30
    odt = {"x": torch.bfloat16, "s8": torch.int8, "f8": torch.float8_e4m3fn}[out]
    y, scales = torch.empty(6, n, dtype=odt, device="cuda"), torch.empty(6, device="cuda")
    hf.rms_norm(x, y, scales=scales if out != "x" else None)
    v = y.float()
    assert bool((v[0] == 0).all())
    if out == "x":
        assert bool(v[1].isnan().all())
        assert bool(v[2, 3].isnan()) and bool((v[2, :3] == 0).all())
    else:
        assert float(scales[0]) == 1.0 and bool(scales[1].isnan()) and bool(scales[2].isnan())
        assert bool((v[1] == 0).all()) if out == "s8" else bool(v[1].isnan().all())
    # sqrt(mean) = 1e-30 is far below eps: out = x / sqrt(eps)
    want = float(x[3, 0]) / math.sqrt(1e-6)
    got = v[3] if out == "x" else v[3] * scales[3]
    assert bool(((got - want).abs() <= want * 2.0 ** -4).all())
    assert bool(v[4:].isfinite().all())
    # eps = 0 on a zero row: 0 * inf
    if out == "x":
        hf.rms_norm(x, y, eps=0.0)
        assert bool(y[0].isnan().all()) and bool(y[4:].isfinite().all())


@pytest.mark.parametrize("out", ["s8", "f8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n", [(6, 40), (6, 1001), (400, 1000), (6, 4096), (6, 40001)])
def test_rms_norm_8_bit_rows_are_the_definitions_quotients(rows, n, dtype, out):
    """Exactly: scales[row] = max|y| / 127 or / 448 and codes y / scale, both one f32 division of the y that the same call
    gives in f32. Rows of subnormal values (whose scale has no reciprocal in f32), of zeros between them, and rows
    whose h * weight underflows or overflows where y does not."""
    a = rnd(1, rows, n)
    a[0] = 0
    a[0, 1:4] = 1e-40, -5e-41, 1e-41
    a[1] *= 1e-38
    a[2] *= 1e-21
    a[3] *= 1e18
    x = torch.from_numpy(a).to(DT[dtype]).cuda()
    top, odt = (127.0, torch.int8) if out == "s8" else (448.0, torch.float8_e4m3fn)
    for wide, eps in ((1.0, 1e-6), (1e-21, 1e-44), (1e25, 0.0), (1e-35, 1e-6)):
        w = torch.from_numpy(np.float32(wide * (1 + rnd(2, n, std=0.1)))).cuda()
        y, q, scales = torch.empty(rows, n, device="cuda"), torch.empty(rows, n, dtype=odt, device="cuda"), torch.empty(rows, device="cuda")
        hf.rms_norm(x, y, weight=w, eps=eps)
        hf.rms_norm(x, q, weight=w, eps=eps, scales=scales)
        yh, codes = y.cpu().numpy(), q.cpu()
        with np.errstate(invalid="ignore", divide="ignore", over="ignore", under="ignore"):
            want = np.abs(yh).max(1) / np.float32(top)  # NaN where the row has one
            want[want == 0] = 1
            t = torch.from_numpy(yh / want[:, None])
        assert np.array_equal(scales.cpu().numpy(), want, equal_nan=True)
        if out == "s8":
            assert torch.equal(codes, t.nan_to_num(0.0).round().clamp(-128, 127).to(torch.int8))
        else:
            t = t.to(torch.float8_e4m3fn).float()
            assert bool(((codes.float() == t) | (codes.float().isnan() & t.isnan())).all())


# ---- gradient ----------------------------------------------------------------------------------------------
def check_grad(rows, n, dtype, dsum=True, weight="x", p=0.0, pitch=0, shift=0, in_place=None, dweight=True, seed=0, w_offset=0.0):
    h, hd = dev(rnd(seed + 1, rows, n, std=2.0), dtype, pitch, shift)
    dy, dyd = dev(rnd(seed + 2, rows, n), dtype, pitch, shift)
    ds, dsd = dev(rnd(seed + 3, rows, n), dtype, pitch, shift) if dsum else (None, None)
    w, wd = dev(1 + rnd(seed + 4, n, std=0.1), dtype if weight == "x" else "f32") if weight else (None, np.ones(n))
    rstd = torch.from_numpy(1.0 / np.sqrt((hd * hd).mean(1) + 1e-6)).float().cuda()
    d = (p, 99 + seed, 1 << 40) if p else None
    dh, dx, dw, edh, edx, edw = ref.rms_norm_backward(dyd, hd, host(rstd), wd, w_offset, dsd, d)
    hb = Band((rows, n), DT[dtype], pitch, shift)
    xb = Band((rows, n), DT[dtype], pitch, shift) if p else None
    out = {None: hb.t, "dy": dy, "h": h, "dsum": ds}[in_place]
    dwt = torch.full((n,), float("nan"), device="cuda") if dweight else None
    ws = Band((hf.rms_norm_workspace_size(rows, n) // 4,), torch.float32) if dweight else None
    hf.rms_norm_backward(dy, h, rstd, out, weight=w, dsum=ds, dx=xb.t if p else None, weight_offset=w_offset,
                         dropout=hf.Dropout(*d) if p else None, dweight=dwt, workspace=ws.t if dweight else None)
    torch.cuda.synchronize()
    what = f"{rows}x{n} {dtype}"
    close(out, dh, edh, dtype, what + " dh")
    if in_place is None:
        hb.check()
    if p:
        xb.check()
        close(xb.t, dx, edx, dtype, what + " dx")
    if dweight:
        ws.check()
        close(dwt, dw, edw, "f32", what + " dweight")
    return dwt


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,n", SHAPES)
def test_rms_norm_backward(rows, n, dtype):
    check_grad(rows, n, dtype)
    check_grad(rows, n, dtype, dsum=False, weight="f32", p=0.3, seed=9, w_offset=1.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pitch,shift", [(8, 0), (3, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("rows,n", [(7, 96), (5, 1001), (3, 4096)])
def test_rms_norm_backward_strides(rows, n, pitch, shift, dtype):
    check_grad(rows, n, dtype, pitch=pitch, shift=shift, p=0.2, weight=None)
    check_grad(rows, n, dtype, pitch=pitch, shift=shift, dweight=False, in_place="dsum")


@pytest.mark.parametrize("n", [96, 1001, 33001])
@pytest.mark.parametrize("in_place", ["dy", "h", "dsum"])
def test_rms_norm_backward_in_place(in_place, n):
    check_grad(9, n, "bf16", in_place=in_place, p=0.1)


@pytest.mark.parametrize("rows,n,dtype", [(640, 64, "f32"), (613, 512, "bf16"), (640, 1024, "f16"), (700, 4096, "bf16"), (611, 4104, "f32"),
                                          (620, 8192, "bf16"), (610, 12000, "bf16"), (609, 16384, "f16"), (609, 16381, "f16"),
                                          (311, 9000, "f32"), (310, 16384, "f32"), (5, 16383, "f32"), (2000, 1001, "bf16")])
def test_rms_norm_backward_of_many_rows(rows, n, dtype):
    """Rows that stream through shared memory: each number of vectors a thread, with and without dsum, weights of
    either type, and a pitch."""
    check_grad(rows, n, dtype, p=0.1)
    check_grad(rows, n, dtype, dsum=False, weight="f32", w_offset=1.0, pitch=64, shift=8)
    check_grad(rows, n, dtype, weight=None, dweight=False, in_place="h")


def test_rms_norm_backward_is_deterministic():
    a = check_grad(1000, 1032, "bf16")
    assert torch.equal(a, check_grad(1000, 1032, "bf16"))


def test_rms_norm_backward_of_no_rows():
    dw = torch.full((8,), 5.0, device="cuda")
    e = torch.empty(0, 8, device="cuda")
    hf.rms_norm_backward(e, e, torch.empty(0, device="cuda"), e, dweight=dw)
    assert bool((dw == 0).all())


@pytest.mark.parametrize("n", [5, 72])
def test_rms_norm_backward_against_differences(n):
    """Central differences of L = sum(dy y) + sum(dsum h) in 64 bits: with a step of 1e-5 their own error is
    below 1e-8, far under the 1e-4 asked for."""
    rows, p, seed = 3, 0.25, 11
    x, r, w = rnd(1, rows, n), rnd(2, rows, n), 1 + rnd(3, n, std=0.1)
    x, r, w, dy, ds = (np.float32(a).astype(np.float64) for a in (x, r, w, rnd(4, rows, n), rnd(5, rows, n)))
    d = (p, seed, 3)

    def loss(x, r, w):
        h, _, y, *_ = ref.rms_norm(x, w, r, d=d)
        return (dy * y).sum() + (ds * h).sum()

    h, rs, *_ = ref.rms_norm(x, w, r, d=d)
    f = lambda a: torch.from_numpy(a).float().cuda()
    dh, dx, dw = (torch.empty(*s, device="cuda") for s in ((rows, n), (rows, n), (n,)))
    ws = torch.empty(hf.rms_norm_workspace_size(rows, n), dtype=torch.uint8, device="cuda")
    hf.rms_norm_backward(f(dy), f(h), f(rs), dh, weight=f(w), dsum=f(ds), dx=dx, dropout=hf.Dropout(*d), dweight=dw,
                         workspace=ws)
    for got, which in ((dx, 0), (dh, 1), (dw, 2)):
        args = [x, r, w]
        base = args[which]
        for at in np.ndindex(*base.shape):
            hi, lo = base.copy(), base.copy()
            hi[at] += 1e-5
            lo[at] -= 1e-5
            num = (loss(*args[:which], hi, *args[which + 1:]) - loss(*args[:which], lo, *args[which + 1:])) / 2e-5
            assert abs(float(got[at]) - num) <= 1e-4 * (1 + abs(num)), (which, at)


# ---- dropout -----------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape,pitch,shift", [((1,), 0, 0), ((7,), 0, 0), ((1000003,), 0, 0), ((1000003,), 0, 1), ((3, 64), 8, 0),
                                               ((5, 77), 0, 0), ((5, 77), 3, 0), ((4, 33, 130), 6, 1), ((70, 4096), 0, 0),
                                               ((70, 4096), 64, 0), ((3, 1002), 2, 2)])
def test_dropout(shape, pitch, shift, dtype):
    for p, seed, offset, res in ((0.1, 3, 0, False), (0.5, (1 << 63) + 12345, (1 << 64) - 1, True)):
        x, xd = dev(rnd(1, *shape), dtype, pitch, shift)
        r, rd = dev(rnd(2, *shape), dtype, pitch, shift) if res else (None, 0.0)
        out = Band(shape, DT[dtype], pitch, shift)
        hf.dropout(x, out.t, hf.Dropout(p, seed, offset), residual=r)
        torch.cuda.synchronize()
        out.check()
        k = ref.keep(p, seed, offset, xd.size).reshape(shape)
        f = np.float32
        want = np.where(k, xd.astype(f) * f(1 / (1 - p)), f(0)) + (rd.astype(f) if res else f(0))
        assert torch.equal(out.t.cpu(), torch.from_numpy(np.ascontiguousarray(want.astype(f))).to(DT[dtype]))


def test_dropout_extremes_and_specials():
    x = torch.tensor([float("nan"), float("inf"), -0.0, 1.0] * 64, device="cuda")
    out = torch.empty_like(x)
    hf.dropout(x, out, hf.Dropout(1.0, 1, 1))
    assert bool((out == 0).all())
    hf.dropout(x, out, hf.Dropout(0.0, 1, 1))
    nan = x.isnan()  # whose bits a multiplication need not keep
    assert torch.equal(out.isnan(), nan) and torch.equal(out[~nan].view(torch.int32), x[~nan].view(torch.int32))
    hf.dropout(x, x, hf.Dropout(0.5, 9, 1))  # in place; a dropped NaN is 0
    k = torch.from_numpy(ref.keep(0.5, 9, 1, 256)).cuda()
    assert bool((x[~k] == 0).all()) and bool((x.isnan() == (k & (torch.arange(256, device="cuda") % 4 == 0))).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,pitch,shift", [(4096, 0, 0), (1001, 0, 0), (72, 3, 1), (40000, 0, 0), (5, 0, 1)])
def test_dropped_elements_of_a_negative_zero_residual(n, pitch, shift, dtype):
    """-0 + 0 is +0, whatever the alignment, in dropout and in the norm's sum; -0 + -0 (a kept element) stays -0."""
    d, rows = hf.Dropout(0.5, 9, 1), 3
    x, _ = dev(np.full((rows, n), -0.0), dtype, pitch, shift)
    r, _ = dev(np.full((rows, n), -0.0), dtype, pitch, shift)
    kept = torch.from_numpy(ref.keep(0.5, 9, 1, rows * n).reshape(rows, n)).cuda()
    out, odd = torch.empty(rows, n, dtype=DT[dtype], device="cuda"), torch.empty(rows, n + 1, dtype=DT[dtype], device="cuda")[:, 1:]
    h, y = Band((rows, n), DT[dtype], pitch, shift).t, torch.empty(rows, n, dtype=DT[dtype], device="cuda")
    for o in (out, odd, Band((rows, n), DT[dtype], pitch, shift).t):
        hf.dropout(x, o, d, residual=r)
        assert bool((o == 0).all()) and torch.equal(o.signbit(), kept)
    for o in (y, Band((rows, n), DT[dtype], pitch, shift).t):
        hf.rms_norm(x, o, residual=r, sum_out=h, dropout=d)
        assert bool((h == 0).all()) and torch.equal(h.signbit(), kept)


def test_dropout_mask_does_not_depend_on_the_shape_and_is_the_norms_mask():
    d = hf.Dropout(0.3, 42, 5)
    x = torch.ones(6, 1001, device="cuda")
    a, b, h, y = (torch.empty_like(x) for _ in range(4))
    hf.dropout(x, a, d)
    hf.dropout(x.view(-1), b.view(-1), d)
    hf.rms_norm(x, y, sum_out=h, dropout=d)
    assert torch.equal(a, b) and torch.equal(a, h)


def test_dropout_state_on_the_device_in_a_graph():
    """A captured call draws a new mask when the state moves on."""
    x, out = torch.ones(4096, device="cuda"), torch.empty(4096, device="cuda")
    state = torch.tensor([17, 100], dtype=torch.int64, device="cuda")
    d = hf.Dropout(0.5, 1, 3, state)
    hf.dropout(x, out, d)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hf.dropout(x, out, d)
        state[1:2].add_(10)
    for step in range(3):
        g.replay()
        k = ref.keep(0.5, 17, 103 + 10 * step, 4096)
        assert np.array_equal(host(out) != 0, k)


# ---- rotary ------------------------------------------------------------------------------------------------
def check_rotary(batch, seq, heads, kv, dim, rot, dtype, interleaved=False, inverse=False, scale=1.0, start=0, packed=False,
                 heads_major=False, in_place=False, shift=0, base=10000.0):
    turns = ref.turns_of(rot, base)
    td = torch.from_numpy(turns.view(np.int64)).cuda()
    pos = (np.arange(seq)[None] + start + 13 * np.arange(batch)[:, None]).astype(np.int32)
    if packed:
        qkv, qkvd = dev(rnd(1, batch, seq, heads + 2 * kv, dim), dtype, 0, shift)
        arrays = [(qkv[:, :, :heads], qkvd[:, :, :heads]), (qkv[:, :, heads:heads + kv], qkvd[:, :, heads:heads + kv])]
    else:
        arrays = [dev(rnd(1, batch, seq, heads, dim), dtype, 0, shift), dev(rnd(2, batch, seq, kv, dim), dtype, 0, shift)]
    bands = []
    for (t, _) in arrays:
        b, s, h, d = t.shape
        if heads_major:
            band = Band((b, h, s, d), DT[dtype], 0, shift)
            band.t = band.t.transpose(1, 2)
        else:
            band = Band((b, s, h, d), DT[dtype], 0, shift)
        bands.append(band)
    outs = [t for t, _ in arrays] if in_place else [b.t for b in bands]
    hf.rotary(arrays[0][0], outs[0], torch.from_numpy(pos).cuda(), td, k=arrays[1][0], k_out=outs[1], interleaved=interleaved,
              inverse=inverse, scale=scale)
    torch.cuda.synchronize()
    for (t, d), o, band in zip(arrays, outs, bands):
        band.check()
        want, err = ref.rotary(d, pos, turns, interleaved, float(np.float32(scale)), inverse)
        close(o, want, err, dtype)
    if packed and in_place:  # the values beside them are untouched
        assert np.array_equal(host(qkv[:, :, heads + kv:]), qkvd[:, :, heads + kv:])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("batch,seq,heads,kv,dim,rot", [(1, 1, 1, 1, 2, 2), (3, 1, 4, 2, 64, 64), (2, 9, 7, 1, 80, 40), (1, 33, 2, 2, 128, 64),
                                                        (2, 5, 3, 3, 10, 6), (1, 4, 40, 8, 128, 128), (1, 3, 2, 1, 256, 0),
                                                        (1, 2, 130, 1, 64, 62), (300, 1, 2, 1, 16, 16), (1, 2, 3, 1, 7, 4),
                                                        (1, 1, 1, 1, 2048, 2048)])
def test_rotary(batch, seq, heads, kv, dim, rot, interleaved, dtype):
    check_rotary(batch, seq, heads, kv, dim, rot, dtype, interleaved, start=1000, packed=True)
    check_rotary(batch, seq, heads, kv, dim, rot, dtype, interleaved, inverse=True, scale=1.25, heads_major=True, start=5)
    check_rotary(batch, seq, heads, kv, dim, rot, dtype, interleaved, packed=True, in_place=True)
    check_rotary(batch, seq, heads, kv, dim, rot, dtype, interleaved, shift=1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,seq,heads,kv,dim,rot", [(2, 2700, 32, 8, 128, 64), (1, 6001, 4, 1, 64, 64), (3, 6700, 2, 1, 16, 8), (1, 5000, 9, 3, 80, 48),
                                                        (1, 2600, 1, 1, 256, 256)])
def test_rotary_of_many_tokens(batch, seq, heads, kv, dim, rot, dtype):
    """Tokens that stream through shared memory, and the same from heads that do not lie together."""
    check_rotary(batch, seq, heads, kv, dim, rot, dtype, True, packed=True, heads_major=True, scale=0.75)
    check_rotary(batch, seq, heads, kv, dim, rot, dtype, False, packed=True, in_place=True, start=7)


def test_rotary_of_many_tokens_with_gaps():
    """One array of strided tokens and, heads first, another whose heads do not lie together."""
    x, xd = dev(rnd(1, 1, 7000, 4, 64), "bf16", 8)  # a pitch of 72 elements from head to head
    turns, pos = ref.turns_of(64), np.arange(7000, dtype=np.int32)[None]
    td, pd = torch.from_numpy(turns.view(np.int64)).cuda(), torch.from_numpy(pos).cuda()
    out = Band((1, 7000, 4, 64), torch.bfloat16, 8)
    hf.rotary(x, out.t, pd, td)
    want, err = ref.rotary(xd, pos, turns)
    out.check()
    close(out.t, want, err, "bf16")
    y = torch.empty(1, 4, 7000, 64, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    y.copy_(x)
    hf.rotary(y, y, pd, td)
    assert torch.equal(y, out.t)


@pytest.mark.parametrize("start", [-5, 500000, 2 ** 31 - 100])
def test_rotary_far_positions(start):
    check_rotary(1, 40, 2, 1, 64, 64, "f32", start=start, base=500000.0)


def test_rotary_inverse_undoes_it_and_positions_repeat():
    x = torch.from_numpy(rnd(1, 2, 6, 4, 64)).float().cuda()
    y, z = torch.empty_like(x), torch.empty_like(x)
    td = torch.from_numpy(hf.rotary_turns(64, scaling="linear", factor=4.0)).cuda()
    pos = torch.arange(6, dtype=torch.int32, device="cuda").expand(2, 6)  # one row for both sequences
    hf.rotary(x, y, pos, td)
    hf.rotary(y, z, pos, td, inverse=True)
    # two rotations, each within 3e-6 (|u| + |v|) of its value (see the reference's bound)
    assert float((x - z).abs().max()) <= 6e-6 * 2 * float(x.abs().max())
    one = torch.empty(6, 4, 64, device="cuda")
    hf.rotary(x[0], one, pos[0], td)  # without a batch dimension
    assert torch.equal(one, y[0])


# ---- logits ------------------------------------------------------------------------------------------------
def check_logits(batch, vocab, dtype, m=0, bias=None, mask=None, penalties=True, out="x", pitch=0, shift=0, in_place=False, seed=0,
                 token=True, special=False, history=None, prompts=True):
    g = np.random.default_rng(seed + 5)
    a = rnd(seed + 1, batch, vocab, std=3.0)
    if special and vocab >= 8:
        a[:, 1], a[0, 2], a[-1, 3], a[:, 4] = np.nan, np.inf, -np.inf, -0.0
    x, xd = dev(a, dtype, pitch, shift)
    kw, args = {}, {}
    if m:
        hist = (g.random((batch, m)) ** 3 * vocab).astype(np.int32)
        hist[g.random((batch, m)) < 0.05] = -1  # padding inside
        hist[0, :1] = vocab  # outside the vocabulary
        if history is not None:
            hist[:] = history
        lens = g.integers(-1, m + 3, batch).astype(np.int32)
        lens[0] = m
        args.update(history=hist, lengths=lens)
        if prompts:
            args["prompts"] = (np.maximum(lens, 0) // 2).astype(np.int32)
        if penalties:
            args.update(repetition=g.uniform(0.8, 1.5, batch).astype(np.float32), frequency=g.uniform(0, 0.5, batch).astype(np.float32),
                        presence=g.uniform(-0.2, 0.5, batch).astype(np.float32))
    for k, v in args.items():
        kw["prompt_lengths" if k == "prompts" else k] = torch.from_numpy(v).cuda()
    if bias:
        b = rnd(seed + 3, *((vocab,) if bias == "row" else (batch, vocab))).astype(np.float32)
        args["bias"], kw["bias"] = b, torch.from_numpy(b).cuda()
    if mask:
        words = (vocab + 31) // 32
        bits = g.integers(0, 1 << 32, (batch, words), dtype=np.uint64).astype(np.uint32)
        bits[0] = 0  # nothing is allowed
        if batch > 1:
            bits[-1] = 0
            bits[-1, -1] = np.uint32(1 << ((vocab - 1) % 32))  # the last token alone
        if mask == "row":
            bits = bits[-1]
        kw["mask"] = torch.from_numpy(bits.view(np.int32)).cuda()
        unpacked = (bits[..., None] >> np.arange(32, dtype=np.uint32)) & 1
        args["allowed"] = unpacked.reshape(*bits.shape[:-1], -1)[..., :vocab].astype(bool)
    odt = DT[dtype] if out == "x" else torch.float32
    ob = Band((batch, vocab), odt, pitch, shift)
    o = x if in_place else ob.t
    tok = torch.full((batch,), -7, dtype=torch.int32, device="cuda") if token else None
    hf.logits_process(x, None if out is None else o, token=tok, **kw)
    torch.cuda.synchronize()
    want, best = ref.logits(xd.astype(np.float32), **args)
    if out is not None:
        ob.check()
        w = torch.from_numpy(want).to(odt)
        got = o.cpu()
        same = (got == w) | (got.isnan() & w.isnan())
        assert bool(same.all()), f"{int((~same).sum())} of {same.numel()} differ"
    if token:
        assert np.array_equal(tok.cpu().numpy(), best), (tok, best)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,vocab", [(1, 1), (2, 5), (3, 33), (4, 1000), (1, 8191), (2, 8192), (3, 8200), (2, 32000), (1, 131072), (2, 50001),
                                         (1, 200003), (300, 260)])
def test_logits(batch, vocab, dtype):
    check_logits(batch, vocab, dtype, m=50, bias="row", mask="rows")
    check_logits(batch, vocab, dtype, m=300, special=True, prompts=False)
    check_logits(batch, vocab, dtype, bias="rows", out="f32", mask="row")
    check_logits(batch, vocab, dtype, m=20, out=None)
    check_logits(batch, vocab, dtype, m=20, in_place=True, token=False, penalties=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pitch,shift", [(8, 0), (3, 0), (0, 1), (5, 3)])
def test_logits_strides(pitch, shift, dtype):
    for vocab in (999, 9000):
        check_logits(5, vocab, dtype, m=40, bias="row", mask="rows", pitch=pitch, shift=shift)
        check_logits(5, vocab, dtype, m=40, mask="rows", pitch=pitch, shift=shift, in_place=True)


def test_logits_many_occurrences_of_one_token():
    """Counts past 16 bits, and a history longer than the vocabulary."""
    check_logits(2, 100, "f32", m=70000, history=7)
    check_logits(2, 100, "f32", m=40000)


@pytest.mark.parametrize("m", [6720, 6800, 9000, 16383, 16384, 66000])
@pytest.mark.parametrize("batch,vocab", [(2, 40000), (3, 150001)])
def test_logits_long_histories(batch, vocab, m):
    """Histories about as long as a table takes (with two blocks an SM and with one), and one whose counts need 32 bits;
    vocabularies of several slabs."""
    check_logits(batch, vocab, "bf16", m=m, bias="row", mask="rows")


@pytest.mark.parametrize("m", [27000, 28000, 32768, 50000, 65535])
@pytest.mark.parametrize("batch,vocab,dtype", [(1, 131072, "bf16"), (1, 200003, "f16"), (64, 65536, "bf16"), (64, 128256, "f32"), (256, 32000, "bf16"),
                                               (256, 50257, "bf16")])
def test_logits_of_wide_history_buffers(batch, vocab, m, dtype):
    """Buffers of 27000 to 65535 entries, whose lists are as large as the counts, over several batches of tokens a block: exact, by
    counting with numpy."""
    g = np.random.default_rng(m + vocab)
    x, xd = dev(rnd(1, batch, vocab, std=3.0), dtype)
    hist = (g.random((batch, m)) ** 3 * vocab).astype(np.int32)
    lens = g.integers(0, m + 1, batch).astype(np.int32)
    lens[0] = m
    prompts = (lens // 2).astype(np.int32)
    rep, fr, pr = (g.uniform(lo, hi, batch).astype(np.float32) for lo, hi in ((0.8, 1.5), (0.0, 0.5), (-0.2, 0.5)))
    out, tok = torch.empty_like(x), torch.empty(batch, dtype=torch.int32, device="cuda")
    c = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    hf.logits_process(x, out, history=c(hist), lengths=c(lens), prompt_lengths=c(prompts), repetition=c(rep), frequency=c(fr),
                      presence=c(pr), token=tok)
    want = xd.astype(np.float32)
    for i in range(batch):
        seen = np.bincount(hist[i, :lens[i]], minlength=vocab) > 0
        count = np.bincount(hist[i, prompts[i]:lens[i]], minlength=vocab)
        l = want[i]
        l = np.where(seen, np.where(l > 0, l / rep[i], l * rep[i]), l)
        l = np.where(seen, l - fr[i] * count.astype(np.float32), l)
        want[i] = np.where(count > 0, l - pr[i], l)
    assert torch.equal(out.cpu(), torch.from_numpy(want).to(DT[dtype]))
    assert np.array_equal(tok.cpu().numpy(), want.argmax(1))


def test_logits_from_two_threads_with_histories_of_two_widths():
    """Calls of one kernel that need different amounts of shared memory, from two host threads at once, each on a stream of
    its own: none is refused, and the tokens are right."""
    import threading

    found = []

    def calls(m):
        with torch.cuda.stream(torch.cuda.Stream()):
            x = torch.zeros(4, 32000, dtype=torch.bfloat16, device="cuda")
            x[:, 77], x[:, 9] = 2.0, 1.0
            hist = torch.full((4, m), 77, dtype=torch.int32, device="cuda")
            pres = torch.full((4,), 1.5, device="cuda")
            tok = torch.zeros(4, dtype=torch.int32, device="cuda")
            try:
                for _ in range(5000):
                    hf.logits_process(x, history=hist, presence=pres, token=tok)
                found.append(tok.tolist())
            except hf.HloError as e:
                found.append(str(e))

    torch.cuda.synchronize()
    threads = [threading.Thread(target=calls, args=(m,)) for m in (8000, 16000)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert found == [[9] * 4] * 2


def test_logits_of_a_full_table():
    """As many different tokens as entries, all of them in one row's slab."""
    g = np.random.default_rng(3)
    hist = np.stack([g.permutation(9000)[:6700] for _ in range(4)]).astype(np.int32)
    check_logits(4, 9000, "f32", m=6700, history=hist, token=True)
    hist = np.stack([g.permutation(700)[:600] for _ in range(400)]).astype(np.int32)
    check_logits(400, 700, "bf16", m=600, history=hist, token=True)


def test_logits_ties_go_to_the_lowest_token():
    x = torch.zeros(2, 70000, device="cuda", dtype=torch.bfloat16)
    x[0, 123] = x[0, 60000] = 4.0
    x[1] = -0.0
    x[1, 17::1000] = 0.0  # -0 and +0 are equal
    tok = torch.empty(2, dtype=torch.int32, device="cuda")
    hf.logits_process(x, token=tok)
    assert tok.tolist() == [123, 0]


def test_logits_of_an_empty_vocabulary():
    tok = torch.full((3,), 5, dtype=torch.int32, device="cuda")
    hf.logits_process(torch.empty(3, 0, device="cuda"), token=tok)
    assert tok.tolist() == [-1, -1, -1]


def test_an_error_is_reported_once():
    """Whatever a call answers, the next one (a kernel whose launch is checked by CUDA's last error) answers for itself, and so does
    torch."""
    x = torch.zeros(1, 131072, dtype=torch.bfloat16, device="cuda")
    try:
        hf.logits_process(x, history=torch.zeros(1, 32768, dtype=torch.int32, device="cuda"),
                          token=torch.empty(1, dtype=torch.int32, device="cuda"))
    except hf.HloError:
        pass
    a = torch.ones(65, device="cuda")
    hf.dropout(a[:64], a[1:].clone(), hf.Dropout(0.5, 1, 2))
    hf.dropout(a[1:], torch.empty(64, device="cuda"), hf.Dropout(0.5, 1, 2))
    torch.cuda.synchronize()


# ---- streams -----------------------------------------------------------------------------------------------
def test_calls_run_on_the_stream_they_are_given():
    """Work queued before on that stream is seen; nothing waits for the default stream."""
    s = torch.cuda.Stream()
    x = torch.zeros(64, 4096, device="cuda")
    y, tok = torch.empty_like(x), torch.empty(64, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        x.fill_(1.0)
        hf.rms_norm(x, y, eps=0.0)
    hf.logits_process(y, token=tok, stream=s)
    s.synchronize()
    assert bool((y == 1.0).all()) and bool((tok == 0).all())


def test_calls_after_another_streams_event():
    """A call that may be set up while the one before it on its stream ends still waits for an event of another stream between
    them, and that stream's next calls for this one's. Powers of two, whose norms are exact."""
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    rows, n = 512, 1024
    d = hf.Dropout(0.0, 1, 1)
    x, y, z, w = (torch.zeros(rows, n, device="cuda") for _ in range(4))
    for step in [2.0 ** (k % 6) for k in range(20)]:
        torch.cuda.synchronize()
        with torch.cuda.stream(b):
            torch.cuda._sleep(200_000)
            z.fill_(step)
            hf.dropout(z, x, d)
            wrote = b.record_event()
        with torch.cuda.stream(a):
            hf.dropout(w, w, d)  # short, and done long before the event
            a.wait_event(wrote)
            hf.dropout(x, y, d, residual=x)
            hf.rms_norm(y, w, eps=0.0)
            read = a.record_event()
        with torch.cuda.stream(b):
            b.wait_event(read)
            hf.dropout(w, x, d, residual=y)
        torch.cuda.synchronize()
        assert bool((y == 2.0 * step).all()) and bool((w == 1.0).all()) and bool((x == 2.0 * step + 1.0).all())


def test_calls_are_captured_into_a_graph():
    """Norm, gradient (two kernels), rotary and logits replayed on new inputs give what direct calls give."""
    rows, n = 700, 1032
    x, r, gy = (torch.from_numpy(rnd(s, rows, n)).to(torch.bfloat16).cuda() for s in (1, 2, 3))
    y, h, dh = (torch.empty_like(x) for _ in range(3))
    rs, dw = torch.empty(rows, device="cuda"), torch.empty(n, device="cuda")
    ws = torch.empty(hf.rms_norm_workspace_size(rows, n), dtype=torch.uint8, device="cuda")
    q = torch.from_numpy(rnd(4, 50, 3, 64)).float().cuda()
    qo = torch.empty_like(q)
    pos, turns = torch.arange(50, dtype=torch.int32, device="cuda"), torch.from_numpy(hf.rotary_turns(64)).cuda()
    hist = torch.arange(rows * 9, dtype=torch.int32, device="cuda").view(rows, 9) % n
    half = torch.full((rows,), 0.5, device="cuda")
    tok = torch.empty(rows, dtype=torch.int32, device="cuda")

    def calls():
        hf.rms_norm(x, y, residual=r, sum_out=h, rstd=rs)
        hf.rms_norm_backward(gy, h, rs, dh, dweight=dw, workspace=ws)
        hf.rotary(q, qo, pos, turns)
        hf.logits_process(y, history=hist, presence=half, token=tok)

    calls()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    x.copy_(torch.from_numpy(rnd(9, rows, n)))
    q.copy_(torch.from_numpy(rnd(8, 50, 3, 64)))
    g.replay()
    got = [t.clone() for t in (y, h, dh, rs, dw, qo, tok)]
    for t in (y, h, dh, rs, dw, qo, tok):
        t.zero_()
    calls()
    assert all(torch.equal(a, b) for a, b in zip(got, (y, h, dh, rs, dw, qo, tok)))


@pytest.mark.parametrize("graph", [False, True])
def test_calls_that_follow_closely_see_each_others_writes(graph):
    """Each call reads or overwrites what the one before it wrote or reads; the device is waited for after every
    call on one side and not at all on the other."""
    rows, heads, dim = 512, 8, 128
    n = heads * dim
    x0, r0 = (torch.from_numpy(rnd(s, rows, n)).float().cuda() for s in (1, 2))
    x, r = x0.clone(), r0.clone()
    h, y, dh = (torch.empty_like(x) for _ in range(3))
    rs, dw = torch.empty(rows, device="cuda"), torch.empty(n, device="cuda")
    ws = torch.empty(hf.rms_norm_workspace_size(rows, n), dtype=torch.uint8, device="cuda")
    pos, turns = torch.arange(rows, dtype=torch.int32, device="cuda"), torch.from_numpy(hf.rotary_turns(dim)).cuda()
    hist = torch.arange(rows * 9, dtype=torch.int32, device="cuda").view(rows, 9) % n
    half = torch.full((rows,), 0.5, device="cuda")
    tok = torch.empty(rows, dtype=torch.int32, device="cuda")
    outs = (x, r, h, y, dh, rs, dw, tok)

    def calls(wait):
        for step in range(5):
            d = hf.Dropout(0.25, 7, 1000 * step)
            hf.rms_norm(x, y, residual=r, sum_out=r, rstd=rs, dropout=d)
            wait()
            hf.rotary(y.view(rows, heads, dim), x.view(rows, heads, dim), pos, turns)
            wait()
            hf.dropout(x, h, d, residual=r)
            wait()
            hf.rms_norm(h, y, rstd=rs)
            wait()
            hf.rms_norm_backward(y, h, rs, dh, dweight=dw, workspace=ws)
            wait()
            hf.rms_norm(dh, x, weight=dw)
            wait()
            hf.logits_process(x, y, history=hist, presence=half, token=tok)
            wait()
            hf.dropout(y, x, d)
            wait()

    calls(torch.cuda.synchronize)
    want = [t.clone() for t in outs]
    run = lambda: calls(lambda: None)
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        run = g.replay
    for _ in range(3):
        x.copy_(x0)
        r.copy_(r0)
        run()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))


# ---- offsets past 32 bits ------------------------------------------------------------------------------------
def _room(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes * 1e9:
        pytest.skip(f"needs {gigabytes} GB of device memory")


def test_dropout_past_2_31_elements():
    _room(16)
    n = (1 << 31) + 4099
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    hf.dropout(x, x, hf.Dropout(0.5, 77, 6))
    for at in (0, (1 << 31) - 64, n - 131):
        first = at // 4 * 4
        words = ref.philox(77, 6, np.arange(first // 4, (at + 131 + 3) // 4)).reshape(-1)[at - first:at - first + 131]
        assert np.array_equal(host(x[at:at + 131]) == 2.0, words >= 1 << 31)


def test_rms_norm_past_2_31_elements():
    _room(32)
    n = 4096
    rows = (1 << 31) // n + 9
    x = torch.ones(rows, n, dtype=torch.bfloat16, device="cuda")
    last, ld = dev(rnd(1, 8, n), "bf16")
    x[-8:] = last
    y = torch.empty_like(x)
    rs = torch.empty(rows, device="cuda")
    hf.rms_norm(x, y, rstd=rs)
    _, r, want, _, er, ey = ref.rms_norm(ld, np.ones(n))
    close(y[-8:], want, ey, "bf16")
    dw = torch.empty(n, device="cuda")
    ws = torch.empty(hf.rms_norm_workspace_size(rows, n), dtype=torch.uint8, device="cuda")
    rs.fill_(1.0)
    hf.rms_norm_backward(x, x, rs, y, dweight=dw, workspace=ws)
    dh, _, _, edh, _, _ = ref.rms_norm_backward(ld, ld, np.ones(8), np.ones(n))
    close(y[-8:], dh, edh, "bf16")
    want = (rows - 8) + (ld * ld).sum(0)
    # ones add exactly up to 2^24; the last rows' products round
    assert np.all(np.abs(host(dw) - want) <= want * 64 * ref.U)


def test_rotary_past_2_31_elements():
    _room(16)
    tokens, heads, dim = (1 << 31) // (64 * 128) + 5, 64, 128
    x = torch.zeros(tokens, heads, dim, dtype=torch.bfloat16, device="cuda")
    last, ld = dev(rnd(1, 4, heads, dim), "bf16")
    x[-4:] = last
    turns = ref.turns_of(dim)
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    hf.rotary(x, x, pos, torch.from_numpy(turns.view(np.int64)).cuda())
    want, err = ref.rotary(ld[None], np.arange(tokens - 4, tokens)[None], turns)
    close(x[-4:], want[0], err[0], "bf16")
    assert bool((x[:2] == 0).all())


def test_rotary_of_the_most_tokens_that_32_bits_count():
    """Rounded up to whole blocks, they are more than 2^31."""
    _room(40)
    tokens, dim = (1 << 31) - 1, 8
    x = torch.zeros(tokens, 1, dim, dtype=torch.bfloat16, device="cuda")
    last, ld = dev(rnd(1, 300, 1, dim), "bf16")
    x[:300], x[-300:] = last, last
    turns = ref.turns_of(dim)
    pos = torch.full((1, 1), 1000, dtype=torch.int32, device="cuda").expand(tokens, 1)  # repeated over the batch
    hf.rotary(x[:, None], x[:, None], pos, torch.from_numpy(turns.view(np.int64)).cuda())
    want, err = ref.rotary(ld[None], np.full((1, 300), 1000), turns)
    close(x[:300], want[0], err[0], "bf16")
    close(x[-300:], want[0], err[0], "bf16")


def test_logits_past_2_31_elements():
    _room(16)
    vocab = 131072
    batch = (1 << 31) // vocab + 3
    x = torch.zeros(batch, vocab, dtype=torch.bfloat16, device="cuda")
    x[-1, 70000], x[-2, 5] = 3.0, 1.0
    hist = torch.full((batch, 2), 5, dtype=torch.int32, device="cuda")
    pres = torch.full((batch,), 2.0, device="cuda")
    tok = torch.empty(batch, dtype=torch.int32, device="cuda")
    hf.logits_process(x, x, history=hist, presence=pres, token=tok)
    assert tok[-3:].tolist() == [0, 0, 70000] and int(tok.sum()) == 70000
    assert float(x[-2, 5]) == -1.0 and float(x[-1, 5]) == -2.0 and float(x[-1, 70000]) == 3.0


# ---- together ----------------------------------------------------------------------------------------------
def test_a_layers_path_forward_and_backward():
    """norm -> product -> rotary -> (a stand-in product) -> dropout, residual and norm, and back, against the
    same path in 64 bits through torch's own differentiation."""
    rows, n, heads, dim = 12, 64, 4, 16
    f = lambda s, *shape, std=1.0: torch.from_numpy(np.float32(rnd(s, *shape, std=std))).cuda()
    x, w1, w2, wq, gout = f(1, rows, n), 1 + f(2, n, std=0.1), 1 + f(3, n, std=0.1), f(4, n, n, std=0.1), f(5, rows, n)
    d = (0.2, 31, 4)
    turns = torch.from_numpy(hf.rotary_turns(dim)).cuda()
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    # forward
    y1, r1 = torch.empty_like(x), torch.empty(rows, device="cuda")
    hf.rms_norm(x, y1, weight=w1, rstd=r1)
    q = (y1 @ wq).view(rows, heads, dim)
    qr = torch.empty_like(q)
    hf.rotary(q, qr, pos, turns)
    h, y2, r2 = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda")
    hf.rms_norm(qr.view(rows, n), y2, weight=w2, residual=x, sum_out=h, rstd=r2, dropout=hf.Dropout(*d))
    # backward
    ws = torch.empty(hf.rms_norm_workspace_size(rows, n), dtype=torch.uint8, device="cuda")
    dh, dqr, dw2, dq, dx, dw1 = (torch.empty_like(t) for t in (x, x, w2, x, x, w1))
    hf.rms_norm_backward(gout, h, r2, dh, weight=w2, dx=dqr, dropout=hf.Dropout(*d), dweight=dw2, workspace=ws)
    hf.rotary(dqr.view(rows, heads, dim), dq.view(rows, heads, dim), pos, turns, inverse=True)
    hf.rms_norm_backward(dq @ wq.t(), x, r1, dx, weight=w1, dsum=dh, dweight=dw1, workspace=ws)
    # the same in 64 bits
    X, W1, W2 = (t.detach().cpu().double().requires_grad_(True) for t in (x, w1, w2))
    WQ, G = wq.cpu().double(), gout.cpu().double()
    norm = lambda t, w: t / (t.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * w
    ang = torch.arange(rows).double()[:, None] * torch.tensor([10000.0 ** (-2 * i / dim) for i in range(dim // 2)]).double()
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    Q = (norm(X, W1) @ WQ).view(rows, heads, dim)
    a, b = Q[..., :dim // 2], Q[..., dim // 2:]
    QR = torch.cat([a * c - b * s, b * c + a * s], -1).reshape(rows, n)
    k = torch.from_numpy(ref.keep(*d, rows * n).reshape(rows, n)).double()
    Y2 = norm(X + QR * k * ref.drop_scale(d[0]), W2)
    Y2.backward(G)
    for got, want in ((y2, Y2), (dx, X.grad), (dw1, W1.grad), (dw2, W2.grad)):
        want = want.detach()
        # a chain of five f32 operators and two products of 64 terms
        assert float((got.cpu().double() - want).abs().max()) <= 2e-5 * (1 + float(want.abs().max()))
