"""Differentiable forms of the sequence operators, and two layers made of them:
projection, gated linear recurrence (``RecurrentLayer``) or queries' and keys'
norms and gated delta rule (``DeltaLayer``), group normalisation with SiLU,
projection. The layers run over whole series (training, prompts) and one time
step at a time against a cache of states (streams)."""

from __future__ import annotations

import torch
from torch import nn

from . import delta, sequence


def _rows(t):
    """A gradient as the kernels take it: channels contiguous."""
    return t if t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


def _field_rows(t):
    """The same for a field, whose rows have to be evenly spaced as well: a sum over an axis hands back a gradient
    expanded over it, a transpose one with its axes in another order."""
    t = _rows(t)
    try:
        sequence._samples(t)
    except ValueError:
        return t.contiguous()
    return t


class _Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, h0, decay, drive, lengths, offsets):
        h, last, carries = sequence.recurrence(x, gate, h0, decay=decay, drive=drive, lengths=lengths,
                                               offsets=offsets, save=True)
        ctx.save_for_backward(x, gate, h0, carries, lengths, offsets)
        ctx.kinds = {"decay": decay, "drive": drive}
        ctx.set_materialize_grads(False)
        return h, last

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh, dlast):
        x, gate, h0, carries, lengths, offsets = ctx.saved_tensors
        if dh is None:
            dh = torch.zeros_like(x, memory_format=torch.contiguous_format)
        dx, dgate, dh0 = sequence.recurrence_backward(
            _rows(dh), x, gate, carries, h0, None if dlast is None else dlast.contiguous(), lengths=lengths,
            offsets=offsets, **ctx.kinds)
        return dx, dgate, dh0 if h0 is not None else None, None, None, None, None


class _GroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, groups, weight, bias, eps, activation, lengths):
        y, stats = sequence.group_norm(x, groups, weight, bias, eps=eps, activation=activation, lengths=lengths,
                                       save=True)
        ctx.save_for_backward(x, stats, weight, bias, lengths)
        ctx.how = groups, activation
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, stats, weight, bias, lengths = ctx.saved_tensors
        groups, activation = ctx.how
        dx, dw, db = sequence.group_norm_backward(_field_rows(dy), x, stats, groups, weight, bias, activation=activation,
                                                  lengths=lengths)
        return dx, None, dw if weight is not None else None, db if bias is not None else None, None, None, None


class _DeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, gate, beta, h0, decay, rate, scale, lengths, offsets):
        ctx.kinds = {"decay": decay, "rate": rate, "scale": scale}
        y, last, carries = delta.delta_rule(q, k, v, gate, beta, h0, lengths=lengths, offsets=offsets, save=True,
                                            **ctx.kinds)
        ctx.save_for_backward(q, k, v, gate, beta, h0, carries, lengths, offsets)
        ctx.set_materialize_grads(False)
        return y, last

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dlast):
        q, k, v, gate, beta, h0, carries, lengths, offsets = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros_like(v, memory_format=torch.contiguous_format)
        *grads, dh0 = delta.delta_rule_backward(
            _rows(dy), q, k, v, gate, beta, carries, h0, None if dlast is None else dlast.contiguous(),
            lengths=lengths, offsets=offsets, **ctx.kinds)
        return *grads, dh0 if h0 is not None else None, None, None, None, None, None


class _QKNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, frequencies, positions, lengths, how):
        ctx.save_for_backward(q, k, q_weight, k_weight, frequencies, positions, lengths)
        ctx.how = how
        ctx.set_materialize_grads(False)
        return delta.qk_norm(q, k, q_weight, k_weight, frequencies=frequencies, positions=positions, lengths=lengths,
                             **how)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dqy, dky):
        q, k, q_weight, k_weight, frequencies, positions, lengths = ctx.saved_tensors
        dqy, dky = (None if x is None else torch.zeros_like(x, memory_format=torch.contiguous_format) if d is None
                    else _rows(d) for d, x in ((dqy, q), (dky, k)))
        grads = delta.qk_norm_backward(dqy, dky, q, k, q_weight, k_weight, frequencies=frequencies,
                                       positions=positions, lengths=lengths, **ctx.how)
        return *grads, None, None, None, None


def recurrence(x, gate, h0=None, *, decay="sigmoid", drive="complement", lengths=None, offsets=None):
    """``sequence.recurrence`` with gradients for x, gate and h0; returns (h, last states)."""
    return _Recurrence.apply(x, gate, h0, decay, drive, lengths, offsets)


def group_norm(x, groups, weight=None, bias=None, *, eps=1e-5, activation=None, lengths=None):
    """``sequence.group_norm`` with gradients for x, weight and bias."""
    return _GroupNorm.apply(x, groups, weight, bias, eps, activation, lengths)


def delta_rule(q, k, v, gate, beta, h0=None, *, decay="sigmoid", rate="sigmoid", scale=None, lengths=None,
               offsets=None):
    """``delta.delta_rule`` with gradients for q, k, v, gate, beta and h0; returns (y, last states)."""
    return _DeltaRule.apply(q, k, v, gate, beta, h0, decay, rate, scale, lengths, offsets)


def qk_norm(q, k=None, q_weight=None, k_weight=None, *, norm="rms", eps=1e-6, frequencies=None, positions=None,
            pairs="halves", lengths=None):
    """``delta.qk_norm`` with gradients for q, k and the weights."""
    return _QKNorm.apply(q, k, q_weight, k_weight, frequencies, positions, lengths,
                         {"norm": norm, "eps": eps, "pairs": pairs})


class RecurrentLayer(nn.Module):
    """y = out(silu(norm(h))) + skip(h), h the recurrence of (x', gate) = in(x)
    over time; each time step is normalised by itself. Inputs [batch, steps,
    inputs], outputs [batch, steps, outputs]. Moved to a 16-bit type
    (``layer.bfloat16()``) or under autocast the fields are of that type; states
    and the normalisation's arithmetic stay float32."""

    def __init__(self, inputs: int, channels: int, outputs: int, groups: int = 8, device="cuda"):
        super().__init__()
        if channels % groups:
            raise ValueError(f"groups must divide the channels: got {groups} for {channels}")
        self.channels, self.groups = channels, groups
        self.into = nn.Linear(inputs, 2 * channels, device=device)
        self.out = nn.Linear(channels, outputs, device=device)
        self.skip = nn.Linear(channels, outputs, bias=False, device=device)
        self.weight = nn.Parameter(torch.ones(channels, device=device))
        self.bias = nn.Parameter(torch.zeros(channels, device=device))
        with torch.no_grad():  # memories from one step to a few hundred
            self.into.bias[channels:] = torch.linspace(-2.0, 6.0, channels, device=device)

    def _norm(self, h):
        return sequence.group_norm(h, self.groups, self.weight.float(), self.bias.float(), activation="silu")

    def forward(self, x, state=None, lengths=None):
        """(y, last states); ``state``: float32 [batch, channels] or None."""
        p = self.into(x)
        h, last = recurrence(p[..., :self.channels], p[..., self.channels:], state, lengths=lengths)
        z = self._norm(h.flatten(0, 1))
        return self.out(z.view_as(h)) + self.skip(h), last

    @torch.no_grad()
    def step(self, x, state, slots=None):
        """One time step: x [batch, inputs]; ``state``, float32 [places,
        channels], moves on in place. Returns y [batch, outputs]."""
        p = self.into(x)
        h = sequence.recurrence_step(p[:, :self.channels], p[:, self.channels:], state, slots)
        return self.out(self._norm(h)) + self.skip(h)


class DeltaLayer(nn.Module):
    """y = out(silu(norm(o))) + skip(x), o the delta rule of (q, k, v, gate,
    beta) = in(x) over time with unit queries and keys, each head of o
    normalised by itself. ``base``: queries and keys are turned by position,
    pair p at base ** (-2 p / keys) radians a step (None: not at all).
    Inputs [batch, steps, inputs], outputs [batch, steps, outputs]. Moved to a
    16-bit type or under autocast the fields are of that type; states and
    the normalisation's arithmetic stay float32."""

    def __init__(self, inputs: int, heads: int, keys: int, values: int, outputs: int, key_heads: int | None = None,
                 base: float | None = None, device="cuda"):
        super().__init__()
        key_heads = heads if key_heads is None else key_heads
        if key_heads < 1 or heads % key_heads:
            raise ValueError(f"key_heads must divide the heads: got {key_heads} for {heads}")
        self.heads, self.key_heads, self.keys, self.values = heads, key_heads, keys, values
        self.parts = [key_heads * keys, key_heads * keys, heads * values, heads, heads]
        self.into = nn.Linear(inputs, sum(self.parts), device=device)
        self.out = nn.Linear(heads * values, outputs, device=device)
        self.skip = nn.Linear(inputs, outputs, bias=False, device=device)
        self.weight = nn.Parameter(torch.ones(heads * values, device=device))
        self.bias = nn.Parameter(torch.zeros(heads * values, device=device))
        self.base = base
        self.frequencies = self._frequencies(device)
        with torch.no_grad():  # memories from a few steps to a few hundred
            self.into.bias[sum(self.parts[:3]):sum(self.parts[:4])] = torch.linspace(1.0, 6.0, heads, device=device)

    def _frequencies(self, device):
        if self.base is None:
            return None
        return self.base ** (-2.0 / self.keys * torch.arange(self.keys // 2, dtype=torch.float64, device=device))

    def _apply(self, fn, recurse=True):
        """Moves the layer. The frequencies are no buffer, which another type or ``to_empty`` would spoil: they are
        made again on the device that the parameters came to."""
        super()._apply(fn, recurse)
        device = self.into.weight.device
        if self.base is not None and self.frequencies.device != device:
            self.frequencies = self._frequencies(device)
        return self

    def _fields(self, x, positions, lengths=None):
        q, k, v, gate, beta = self.into(x).split(self.parts, -1)
        q, k = (t.unflatten(-1, (self.key_heads, self.keys)) for t in (q, k))
        q, k = delta.qk_norm(q, k, norm="l2", frequencies=self.frequencies, positions=positions, lengths=lengths)
        return q, k, v.unflatten(-1, (self.heads, self.values)), gate, beta

    def _norm(self, y):
        return sequence.group_norm(y.reshape(-1, self.heads * self.values), self.heads,
                                   self.weight.float(), self.bias.float(), activation="silu")

    def forward(self, x, state=None, lengths=None, positions=None):
        """(y, last states); ``state``: float32 [batch, heads, keys, values]
        or None; ``positions``: int32 [batch, steps], None for 0, 1, 2, ..."""
        fields = self._fields(x, positions, lengths)
        y, last = delta.delta_rule(*fields, state, lengths=lengths)
        return self.out(self._norm(y).view(*y.shape[:-2], -1)) + self.skip(x), last

    @torch.no_grad()
    def step(self, x, state, slots=None, positions=None):
        """One time step: x [batch, inputs]; ``state``, float32 [places, heads,
        keys, values], moves on in place; ``positions``: int32 [batch], needed
        where the layer turns by position. Returns y [batch, outputs]."""
        if self.frequencies is not None and positions is None:
            raise ValueError("a layer that turns by position needs the positions of a step")
        y = delta.delta_rule_step(*self._fields(x, positions), state, slots)
        return self.out(self._norm(y)) + self.skip(x)
