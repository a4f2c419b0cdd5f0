"""The layer operators together: the small decoder of transpose_heroes_gb300.decoder serves and trains with
them. The same model written in 64 bits with torch's own operations is the reference."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import layer_reference as ref
import transpose_heroes_gb300 as hf

pytestmark = pytest.mark.gpu

PROMPT = [3, 1, 4, 1, 5, 9, 2, 6, 5, 3, 5]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transpose_heroes_gb300 import build

    build.build()
    hf.lib()


def model(**kw):
    from transpose_heroes_gb300 import decoder

    return decoder.Decoder(vocab=300, width=96, layers=2, heads=4, kv=2, dim=32, hidden=160, **kw)


def reference(m, tokens, p=0.0, seed=0):
    """(logits of every position, the parameters they depend on), in 64 bits on the CPU."""
    D = lambda t: t.detach().double().cpu().requires_grad_(True)  # noqa: E731
    embed, head, last = D(m.embed), D(m.head), D(m.last)
    layers = [{k: D(v) for k, v in w.items()} for w in m.layers]
    tokens = torch.as_tensor(tokens).cpu()
    n, place = len(tokens), [0]

    def drop(x):
        if not p:
            return x
        k = torch.from_numpy(ref.keep(p, seed, place[0], x.numel()).reshape(x.shape)).double()
        place[0] += 1
        return x * k * ref.drop_scale(p)

    norm = lambda t, w: t / (t.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w  # noqa: E731
    angle = torch.arange(n).double()[:, None] * torch.tensor([10000.0 ** (-2 * i / m.dim) for i in range(m.dim // 2)]).double()
    c, s = angle.cos()[:, None], angle.sin()[:, None]

    def turn(x):
        a, b = x[..., :m.dim // 2], x[..., m.dim // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    h = drop(embed[tokens])
    for w in layers:
        qkv = (norm(h, w["n1"]) @ w["qkv"]).view(n, m.heads + 2 * m.kv, m.dim)
        q, k, v = qkv.split([m.heads, m.kv, m.kv], 1)
        k, v = turn(k).repeat_interleave(m.heads // m.kv, 1), v.repeat_interleave(m.heads // m.kv, 1)
        a = torch.einsum("thd,shd->hts", turn(q), k) / math.sqrt(m.dim)
        a = a.masked_fill(torch.ones(n, n).triu(1).bool(), -math.inf).softmax(-1)
        h = h + drop(torch.einsum("hts,shd->thd", a, v).flatten(1) @ w["o"])
        y = norm(h, w["n2"])
        h = h + drop((torch.nn.functional.silu(y @ w["gate"]) * (y @ w["up"])) @ w["down"])
    return norm(h, last) @ head, [embed, head, last] + [t for w in layers for t in w.values()]


def test_prompt_and_single_tokens_agree_with_64_bits():
    """Two layers of f32 products of up to 160 terms and a handful of operators: far inside 1e-4 of the logits'
    size (f32 products of k terms err by at most k 2^-24, here about 1e-5)."""
    m = model()
    want, _ = reference(m, PROMPT)
    scale = float(want.detach().abs().max())
    whole = m.forward(torch.tensor(PROMPT, device="cuda"), [None] * 2, 0)
    assert float((whole[0].cpu().double() - want[-1].detach()).abs().max()) <= 1e-4 * scale
    cache = [None] * 2
    for i, t in enumerate(PROMPT):
        one = m.forward(torch.tensor([t], device="cuda"), cache, i)
        assert float((one[0].cpu().double() - want[i].detach()).abs().max()) <= 1e-4 * scale


def test_generation_is_the_references_greedy_choice():
    m = model()
    got = m.generate(PROMPT, 6, repetition=1.3, frequency=0.2, presence=0.1)
    tokens = list(PROMPT)
    for t in got:
        l = reference(m, tokens)[0][-1].detach().numpy()
        made = tokens[len(PROMPT):]
        for v in set(tokens):
            l[v] = l[v] / np.float32(1.3) if l[v] > 0 else l[v] * np.float32(1.3)
        for v in set(made):
            l[v] -= 0.2 * made.count(v) + 0.1
        top = np.sort(l)[-2:]
        if top[1] - top[0] > 1e-3:  # otherwise f32 may choose either
            assert t == int(l.argmax())
        tokens.append(t)


def test_generation_under_a_mask():
    m = model()
    bits = np.zeros(10, np.uint32)
    for v in (7, 40, 299):
        bits[v // 32] |= np.uint32(1 << (v % 32))
    mask = torch.from_numpy(bits.view(np.int32)).cuda()
    assert set(m.generate(PROMPT, 8, mask=mask)) <= {7, 40, 299}
    assert m.generate(PROMPT, 8, mask=torch.zeros_like(mask)) == []


@pytest.mark.parametrize("p", [0.0, 0.2])
def test_training_gradients_agree_with_64_bits(p):
    m = model()
    for t in m.parameters():
        t.requires_grad_(True)
    tokens = torch.tensor(PROMPT, device="cuda")
    loss = m.loss(tokens, p=p, seed=5)
    loss.backward()
    logits, params = reference(m, PROMPT[:-1], p, 5)
    want = torch.nn.functional.cross_entropy(logits, tokens[1:].cpu())
    want.backward()
    assert abs(float(loss.detach()) - float(want.detach())) <= 1e-4 * (1 + abs(float(want.detach())))
    for got, w in zip(m.parameters(), params):
        # back through two layers the f32 errors of a dozen products add up: still under 1e-3 of the gradient's size
        assert float((got.grad.cpu().double() - w.grad).abs().max()) <= 1e-3 * float(w.grad.abs().max())


def test_training_learns():
    m = model()
    for t in m.parameters():
        t.requires_grad_(True)
    opt = torch.optim.Adam(m.parameters(), lr=2e-3)
    tokens = torch.tensor([3, 1, 4, 1, 5, 9, 2, 6] * 6, device="cuda")
    first = float(m.loss(tokens).detach())
    for step in range(30):
        opt.zero_grad()
        m.loss(tokens, p=0.1, seed=step).backward()
        opt.step()
    assert float(m.loss(tokens).detach()) < 0.2 * first
    assert m.generate([3, 1, 4, 1, 5, 9, 2, 6, 3, 1], 6) == [4, 1, 5, 9, 2, 6]


# ---- the differentiable forms ------------------------------------------------------------------------------
def _layouts(shape):
    """The same values dense, transposed, and with a gap after every element."""
    a = torch.randn(*shape, generator=torch.Generator().manual_seed(3)).cuda()
    gaps = torch.zeros(*shape[:-1], 2 * shape[-1], device="cuda")[..., ::2]
    gaps.copy_(a)
    return [a, a.transpose(0, -1).contiguous().transpose(0, -1), gaps]


FORMS = {
    "drop": lambda D, x: D.drop(x, hf.Dropout(0.5, 3, 4)),
    "rotate": lambda D, x: D.rotate(x, torch.arange(5, dtype=torch.int32, device="cuda"), torch.from_numpy(hf.rotary_turns(8)).cuda()),
    "norm": lambda D, x: D.rms_norm_residual(x, torch.arange(1.0, 17.0, device="cuda")[::2])[0],
    "residual": lambda D, x: D.rms_norm_residual(torch.ones(5, 3, 8, device="cuda"), torch.ones(8, device="cuda"), x)[0],
}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("reduce", ["sum", "mean", "transposed", "column"])
def test_differentiable_forms_take_any_strides(form, reduce):
    """Inputs and gradients that are transposed, strided or expanded (of sum and mean) give what dense ones give."""
    from transpose_heroes_gb300 import decoder as D

    weigh = torch.randn(8, 3, 5, generator=torch.Generator().manual_seed(4)).cuda()
    results = []
    for x in _layouts((5, 3, 8)):
        for dense in (True, False):
            x = x.detach().requires_grad_(True)
            y = FORMS[form](D, x)
            if dense:  # the gradient passes through a dense copy
                y = y * torch.ones_like(y)
            loss = {"sum": lambda: y.sum(), "mean": lambda: y.mean(), "transposed": lambda: (y.transpose(0, 2) * weigh).sum(),
                    "column": lambda: y[..., 2].sum()}[reduce]()
            loss.backward()
            results.append((y.detach(), x.grad))
    for y, g in results[1:]:
        assert torch.equal(y, results[0][0]) and torch.equal(g, results[0][1])


def test_a_norm_without_weight_or_with_a_fixed_one():
    """No weight, and one that wants no gradient, leave the gradient of x what it is."""
    from transpose_heroes_gb300 import decoder as D

    base = torch.randn(5, 8, generator=torch.Generator().manual_seed(3)).cuda()
    grads = []
    for weight in (torch.ones(8, device="cuda", requires_grad=True), torch.ones(8, device="cuda"), None):
        x = base.clone().requires_grad_(True)
        D.rms_norm_residual(x, weight)[0].pow(3).sum().backward()
        grads.append(x.grad)
    assert torch.equal(grads[0], grads[1]) and torch.equal(grads[0], grads[2])


@pytest.mark.parametrize("form", FORMS)
def test_second_derivatives_raise(form):
    """Not silently left out, where another path carries the graph on."""
    from transpose_heroes_gb300 import decoder as D

    x = torch.randn(5, 3, 8, generator=torch.Generator().manual_seed(3)).cuda().requires_grad_(True)
    g, = torch.autograd.grad(FORMS[form](D, x).pow(2).sum() + x.pow(3).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


def test_overwriting_a_saved_tensor_is_noticed():
    """The sum h that the norm keeps for its backward pass is the caller's residual stream: a call that writes over it moves its
    version, as torch's own operations do, and the backward pass raises in place of using the new values."""
    from transpose_heroes_gb300 import decoder as D

    x = torch.randn(5, 8, device="cuda", requires_grad=True)
    y, h = D.rms_norm_residual(x, torch.ones(8, device="cuda"))
    with torch.no_grad():
        hf.dropout(h, h, hf.Dropout(0.5, 1, 2))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_every_output_moves_its_version():
    new = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    x, out, s, r = new(4, 8), new(4, 8), new(4, 8), new(4)
    q, scales, ws, dw, dx = new(4, 8, t=torch.int8), new(4), new(1 << 16, t=torch.uint8), new(8), new(4, 8)
    hf.rms_norm(x, out, sum_out=s, rstd=r)
    hf.rms_norm(x, q, scales=scales)
    hf.rms_norm_backward(x, s, r, out, dx=dx, dropout=hf.Dropout(0.5), dweight=dw, workspace=ws)
    a, b, tok, l = new(3, 2, 8), new(3, 1, 8), new(4, t=torch.int32), new(4, 8)
    turns = new(4, t=torch.int64)
    hf.rotary(a, a, new(3, t=torch.int32), turns, k=b, k_out=b)
    hf.logits_process(x, l, token=tok)
    hf.dropout(x, l, hf.Dropout(0.5))
    assert [t._version for t in (x, out, s, r, q, scales, ws, dw, dx, a, b, tok, l, turns)] == [0, 2, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 2, 0]
    with torch.inference_mode():  # tensors that have no versions
        hf.dropout(x, torch.empty_like(x), hf.Dropout(0.5))
    with pytest.raises(hf.HloError):
        hf.dropout(x, x[:, 1:], hf.Dropout(0.5))  # refused: nothing was written
    assert x._version == 0
