"""The layer operators in use: differentiable forms for training, and a small decoder that serves and trains
with them (matrix products and attention itself are plain torch).

    python -m transpose_heroes_gb300.decoder     # trains a few steps on a toy text, then continues it

    rms_norm_residual(x, weight, residual, dropout)   y, h: h = residual + drop(x), y = rms_norm(h) * weight
    rotate(x, positions, turns)                       rotary positions
    drop(x, params)                                   dropout whose mask is never stored

Their gradients are not differentiable again: a second derivative through them raises.
"""

from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

from . import Dropout
from . import dropout as _dropout
from . import logits_process, rms_norm, rms_norm_backward, rms_norm_workspace_size, rotary, rotary_turns


def _rows(t):
    """t, copied only where the elements of a row do not lie together (a transposed or expanded tensor)."""
    return t if t is None or t.dim() == 0 or t.shape[-1] <= 1 or t.stride(-1) == 1 else t.contiguous()


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, dropout, eps):
        x, residual, weight = x.contiguous(), _rows(residual), None if weight is None else weight.contiguous()
        y, h = torch.empty_like(x), torch.empty_like(x)
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rms_norm(x, y, weight=weight, residual=residual, sum_out=h, rstd=rstd, eps=eps, dropout=dropout)
        ctx.save_for_backward(h, weight, rstd)
        ctx.dropout, ctx.joined = dropout, residual is not None
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dsum):
        h, weight, rstd = ctx.saved_tensors
        n = h.shape[-1]
        dh = torch.empty_like(h)
        dx = torch.empty_like(h) if ctx.dropout is not None else None
        dw = ws = None
        if ctx.needs_input_grad[1]:
            dw = torch.empty(n, dtype=torch.float32, device=h.device)
            ws = torch.empty(rms_norm_workspace_size(h.numel() // n, n), dtype=torch.uint8, device=h.device)
        rms_norm_backward(dy.contiguous(), h, rstd, dh, weight=weight, dsum=dsum.contiguous(), dx=dx, dropout=ctx.dropout,
                          dweight=dw, workspace=ws)
        return dx if dx is not None else dh, None if dw is None else dw.to(weight.dtype), dh if ctx.joined else None, None, None


def rms_norm_residual(x, weight, residual=None, dropout=None, eps=1e-6):
    """(y, h): h = residual + drop(x), y = h / rms(h) * weight (None: ones); differentiable in x, weight and residual."""
    return _RmsNorm.apply(x, weight, residual, dropout, eps)


class _Rotate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, positions, turns, interleaved, scale):
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        rotary(_rows(x), out, positions, turns, interleaved=interleaved, scale=scale)
        ctx.save_for_backward(positions, turns)
        ctx.how = interleaved, scale
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        positions, turns = ctx.saved_tensors
        out = torch.empty(g.shape, dtype=g.dtype, device=g.device)
        rotary(_rows(g), out, positions, turns, interleaved=ctx.how[0], scale=ctx.how[1], inverse=True)
        return out, None, None, None, None


def rotate(x, positions, turns, interleaved=False, scale=1.0):
    """rotary() on [batch, seq, heads, dim] or [seq, heads, dim]; differentiable in x."""
    return _Rotate.apply(x, positions, turns, interleaved, scale)


class _Drop(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, params):
        ctx.params = params
        return _dropout(_rows(x), torch.empty(x.shape, dtype=x.dtype, device=x.device), params)

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        return _dropout(_rows(g), torch.empty(g.shape, dtype=g.dtype, device=g.device), ctx.params), None


def drop(x, params):
    """drop(x) for params = Dropout(p, seed, offset); the backward pass makes the mask again."""
    return _Drop.apply(x, params)


class Decoder:
    """A decoder of pre-norm layers: attention with rotary positions and shared key heads, and a gated
    feed-forward block; dropout on what each block adds to the residual stream."""

    def __init__(self, vocab=512, width=256, layers=2, heads=4, kv=2, dim=64, hidden=512, dtype=torch.float32, seed=0,
                 device="cuda"):
        g = torch.Generator(device="cpu").manual_seed(seed)
        self.vocab, self.width, self.heads, self.kv, self.dim = vocab, width, heads, kv, dim

        def matrix(*shape):
            return (torch.randn(*shape, generator=g) / math.sqrt(shape[0])).to(device=device, dtype=dtype)

        one = lambda: torch.ones(width, dtype=dtype, device=device)  # noqa: E731
        self.embed = torch.randn(vocab, width, generator=g).to(device=device, dtype=dtype)
        self.head, self.last = matrix(width, vocab), one()
        self.layers = [dict(n1=one(), qkv=matrix(width, (heads + 2 * kv) * dim), o=matrix(heads * dim, width), n2=one(),
                            gate=matrix(width, hidden), up=matrix(width, hidden), down=matrix(hidden, width))
                       for _ in range(layers)]
        self.turns = torch.from_numpy(rotary_turns(dim)).to(device)

    def parameters(self):
        return [self.embed, self.head, self.last] + [t for layer in self.layers for t in layer.values()]

    def _attend(self, q, k, v, first):
        """q [t, heads, dim] at positions first .. first + t - 1 over k, v [length, kv, dim]."""
        share = self.heads // self.kv
        k, v = k.repeat_interleave(share, 1), v.repeat_interleave(share, 1)
        s = torch.einsum("thd,shd->hts", q, k) / math.sqrt(self.dim)
        seen = torch.arange(k.shape[0], device=q.device) <= torch.arange(first, first + q.shape[0], device=q.device)[:, None]
        return torch.einsum("hts,shd->thd", s.masked_fill(~seen, -math.inf).softmax(-1), v).flatten(1)

    # ---- serving -------------------------------------------------------------------------------------------
    @torch.no_grad()
    def forward(self, tokens, cache, first):
        """The last position's logits [1, vocab] for `tokens` at positions first ..; cache: per layer (k, v) so far,
        extended in place. The residual stream h is updated in place by each norm."""
        h = self.embed[tokens].clone()
        positions = torch.arange(first, first + len(tokens), dtype=torch.int32, device=h.device)
        y, added = torch.empty_like(h), None
        for i, w in enumerate(self.layers):
            if added is None:
                rms_norm(h, y, weight=w["n1"])
            else:
                rms_norm(added, y, weight=w["n1"], residual=h, sum_out=h)
            qkv = (y @ w["qkv"]).view(len(tokens), self.heads + 2 * self.kv, self.dim)
            q, k, v = qkv.split([self.heads, self.kv, self.kv], 1)
            rotary(q, q, positions, self.turns, k=k, k_out=k)  # in place, in the packed projection
            cache[i] = (k, v) if cache[i] is None else tuple(torch.cat(p) for p in zip(cache[i], (k, v)))
            added = self._attend(q, *cache[i], first) @ w["o"]
            rms_norm(added, y, weight=w["n2"], residual=h, sum_out=h)
            added = (torch.nn.functional.silu(y @ w["gate"]) * (y @ w["up"])) @ w["down"]
        rms_norm(added, y, weight=self.last, residual=h, sum_out=h)
        return y[-1:] @ self.head

    @torch.no_grad()
    def generate(self, prompt, count, repetition=1.0, frequency=0.0, presence=0.0, mask=None):
        """`count` greedy tokens after `prompt` (a list); mask: s32 bits of the allowed tokens, or None. Stops early
        when the mask leaves nothing."""
        dev = self.embed.device
        history = torch.zeros(1, len(prompt) + count, dtype=torch.int32, device=dev)
        history[0, :len(prompt)] = torch.tensor(prompt, dtype=torch.int32)
        vector = lambda x, t: torch.tensor([x], dtype=t, device=dev)  # noqa: E731
        length, prompts = vector(len(prompt), torch.int32), vector(len(prompt), torch.int32)
        terms = [vector(x, torch.float32) for x in (repetition, frequency, presence)]
        token = vector(-1, torch.int32)
        cache, tokens, first = [None] * len(self.layers), list(prompt), 0
        step = torch.tensor(tokens, device=dev)
        while len(tokens) < len(prompt) + count:
            logits = self.forward(step, cache, first)
            logits_process(logits, history=history, lengths=length, prompt_lengths=prompts, repetition=terms[0],
                           frequency=terms[1], presence=terms[2], mask=mask, token=token)
            first = len(tokens)
            new = int(token)
            if new < 0:
                break
            history[0, first] = new
            length += 1
            tokens.append(new)
            step = torch.tensor([new], device=dev)
        return tokens[len(prompt):]

    # ---- training ------------------------------------------------------------------------------------------
    def loss(self, tokens, p=0.0, seed=0):
        """Mean cross entropy of each next token; p: dropout, a new mask for every (seed, place)."""
        n = len(tokens) - 1
        positions = torch.arange(n, dtype=torch.int32, device=tokens.device)
        mask = iter(Dropout(p, seed, k) if p else None for k in range(2 * len(self.layers) + 1))
        h = self.embed[tokens[:-1]]
        if p:
            h = drop(h, next(mask))
        y, h = rms_norm_residual(h, self.layers[0]["n1"])
        for i, w in enumerate(self.layers):
            qkv = (y @ w["qkv"]).view(n, self.heads + 2 * self.kv, self.dim)
            q, k, v = qkv.split([self.heads, self.kv, self.kv], 1)
            q, k = rotate(q, positions, self.turns), rotate(k, positions, self.turns)
            y, h = rms_norm_residual(self._attend(q, k, v, 0) @ w["o"], w["n2"], h, next(mask) if p else None)
            added = (torch.nn.functional.silu(y @ w["gate"]) * (y @ w["up"])) @ w["down"]
            after = self.layers[i + 1]["n1"] if i + 1 < len(self.layers) else self.last
            y, h = rms_norm_residual(added, after, h, next(mask) if p else None)
        return torch.nn.functional.cross_entropy((y @ self.head).float(), tokens[1:])


def main():
    model = Decoder()
    text = torch.tensor(([3, 1, 4, 1, 5, 9, 2, 6] * 12), device="cuda")
    for t in model.parameters():
        t.requires_grad_(True)
    opt = torch.optim.Adam(model.parameters(), lr=2e-3)
    for step in range(30):
        opt.zero_grad()
        loss = model.loss(text, p=0.1, seed=step)
        loss.backward()
        opt.step()
        if step % 10 == 9:
            print(f"step {step + 1}: loss {float(loss.detach()):.4f}")
    print("continues 3 1 4 1 5 with", model.generate([3, 1, 4, 1, 5], 8))
    print("and penalised for repeating itself:", model.generate([3, 1, 4, 1, 5], 8, frequency=100.0))


if __name__ == "__main__":
    main()
