"""What the Python binding of the layer operators refuses of tensors on the GPU. The injected fault answers in place of every
launch, so nothing that should have been refused reaches the device."""

import pytest

torch = pytest.importorskip("torch")

import transpose_heroes_gb300 as hf

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transpose_heroes_gb300 import build

    build.build()
    hf.lib()


@pytest.fixture(autouse=True)
def no_launch(monkeypatch):
    monkeypatch.setenv("HLOFUSION_FAULT", "all")


def refused(call, word=""):
    with pytest.raises(hf.HloError) as e:
        call()
    assert e.value.status == 1 and word in str(e.value), str(e.value)


def accepted(call):
    with pytest.raises(hf.HloError) as e:
        call()
    assert e.value.status == 3 and "injected fault" in str(e.value), str(e.value)


def zeros(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


OTHER = [torch.float64, torch.int64, torch.uint8, torch.int16, torch.bool]


@pytest.mark.parametrize("dtype", OTHER)
def test_weights_of_another_type(dtype):
    """Neither the input's type nor f32: never read as one of them."""
    w = zeros(8, dtype=dtype)
    x, y = zeros(4, 8), zeros(4, 8)
    refused(lambda: hf.rms_norm(x, y, weight=w), "weight")
    refused(lambda: hf.rms_norm(x, y, weight=w, weight_dtype="bf16"), "weight")
    refused(lambda: hf.rms_norm_backward(x, y, zeros(4), zeros(4, 8), weight=w), "weight")
    refused(lambda: hf.rms_norm(x, y, weight=zeros(8, dtype=torch.bfloat16)), "weight type")
    accepted(lambda: hf.rms_norm(x, y, weight=zeros(8)))
    accepted(lambda: hf.rms_norm(zeros(4, 8, dtype=torch.bfloat16), zeros(4, 8, dtype=torch.bfloat16), weight=zeros(8)))


@pytest.mark.parametrize("dtype", [torch.float64, torch.float32, torch.int32, torch.uint8, torch.int16, torch.bool])
def test_turns_of_another_type(dtype):
    """Only 64-bit whole numbers are angles; narrower elements would be read past their end."""
    q, pos = zeros(3, 2, 8), zeros(3, dtype=torch.int32)
    refused(lambda: hf.rotary(q, q, pos, zeros(4, dtype=dtype)), "turns")
    refused(lambda: hf.rotary(q, q, pos, zeros(4, dtype=dtype), n_pairs=4), "turns")
    refused(lambda: hf.rotary(q, q, pos, zeros(8, dtype=torch.int64)[::2]), "turns")
    accepted(lambda: hf.rotary(q, q, pos, zeros(4, dtype=torch.int64)))


def test_more_pairs_than_turns():
    q, pos, turns = zeros(3, 2, 8), zeros(3, dtype=torch.int32), zeros(2, dtype=torch.int64)
    refused(lambda: hf.rotary(q, q, pos, turns, n_pairs=4), "turns has 2")
    refused(lambda: hf.rotary(q, q, pos, turns, n_pairs=3), "turns has 2")
    refused(lambda: hf.rotary(q, q, pos, turns, n_pairs=-(1 << 32)), "pairs")  # not 0 of them
    refused(lambda: hf.rotary(q, q, pos, turns, n_pairs=-1), "pairs")
    for n in (None, 2, 1):
        accepted(lambda: hf.rotary(q, q, pos, turns, n_pairs=n))
    accepted(lambda: hf.rotary(q, q, pos, zeros(4, dtype=torch.int64).data_ptr(), n_pairs=4))


def test_workspaces():
    x, dh, rstd, dw = zeros(4, 8), zeros(4, 8), zeros(4), zeros(8)
    n = hf.rms_norm_workspace_size(4, 8)
    run = lambda ws, **kw: hf.rms_norm_backward(x, x, rstd, dh, dweight=dw, workspace=ws, **kw)  # noqa: E731
    refused(lambda: run(torch.zeros(n, dtype=torch.uint8)), "on the GPU")
    refused(lambda: run(zeros(1, dtype=torch.uint8).expand(n)), "contiguous")
    refused(lambda: run(zeros(2 * n, dtype=torch.uint8)[::2]), "contiguous")
    refused(lambda: run(zeros(8, dtype=torch.uint8), workspace_bytes=n), "the tensor has 8")
    with pytest.raises(hf.HloError) as e:
        run(zeros(n - 1, dtype=torch.uint8))
    assert e.value.status == 4
    with pytest.raises(TypeError):
        run("scratch")
    accepted(lambda: run(zeros(n, dtype=torch.uint8)))
    accepted(lambda: run(zeros(n, dtype=torch.uint8), workspace_bytes=n))
    accepted(lambda: run(zeros((n + 7) // 8, dtype=torch.float64)))
    ws = zeros(n, dtype=torch.uint8)
    accepted(lambda: run(ws.data_ptr(), workspace_bytes=n))


def test_tensors_of_another_device():
    """With one GPU in the machine, tensors without memory that say they are on the next one."""

    class Elsewhere(torch.Tensor):
        __torch_dispatch__ = classmethod(lambda cls, *a, **kw: NotImplemented)

    other = f"cuda:{torch.cuda.current_device() + 1}"
    x, w, scratch = (torch.Tensor._make_wrapper_subclass(Elsewhere, shape, dtype=t, device=other)
                     for shape, t in (((4, 8), torch.float32), ((8,), torch.float32), ((1 << 20,), torch.uint8)))
    a, b = zeros(4, 8), zeros(4, 8)
    for call in (lambda: hf.rms_norm(x, b), lambda: hf.rms_norm(a, x), lambda: hf.rms_norm(a, b, weight=w),
                 lambda: hf.dropout(a, b, hf.Dropout(0.5), residual=x), lambda: hf.logits_process(a, x),
                 lambda: hf.rms_norm_backward(a, a, zeros(4), b, dweight=zeros(8), workspace=scratch)):
        refused(call, f"on {other}")
    accepted(lambda: hf.rms_norm(a, b))


def test_lazily_negated_tensors():
    """A view whose values are the negatives of its memory's."""
    x = torch._neg_view(zeros(4, 8))
    refused(lambda: hf.rms_norm(x, zeros(4, 8)), "negates")
    refused(lambda: hf.rms_norm(zeros(4, 8), x), "negates")
    accepted(lambda: hf.rms_norm(x.resolve_neg(), zeros(4, 8)))
