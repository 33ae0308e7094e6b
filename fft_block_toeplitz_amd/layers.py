"""Differentiable forms of the sequence operators, and a recurrent layer made
of them: projection, gated linear recurrence, group normalisation with SiLU,
projection. The layer runs over whole series (training, prompts) and one time
step at a time against a cache of states (streams)."""

from __future__ import annotations

import torch
from torch import nn

from . import sequence


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


def recurrence(x, gate, h0=None, *, decay="sigmoid", drive="complement", lengths=None, offsets=None):
    """``sequence.recurrence`` with gradients for x, gate and h0; returns (h, last states)."""
    return _Recurrence.apply(x, gate, h0, decay, drive, lengths, offsets)


def group_norm(x, groups, weight=None, bias=None, *, eps=1e-5, activation=None, lengths=None):
    """``sequence.group_norm`` with gradients for x, weight and bias."""
    return _GroupNorm.apply(x, groups, weight, bias, eps, activation, lengths)


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
