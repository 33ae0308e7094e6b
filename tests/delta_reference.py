"""The gated delta rule and the norms of its queries and keys from their
definitions in float64, step by step, and how far float32 arithmetic may be off.

Tolerances are norms relative to norms, for one sequence and head at a time.
An FP32 result goes through sums over up to 128 keys and three times 64 steps in
one run, and the states of earlier runs reach it through factors below one: some
400 roundings of 2^-24 of either sign, sqrt(400) = 20 of them, three times that
and a little: 64. A 16-bit result comes from products that are kept to 2^-16,
eight of them one behind the other at most: 2^-13, and is rounded once, by half
a step at most. Each row by itself may be off by 8 times as much of its own norm
and the rows' mean: rows are parts of what the sums above go over."""
import torch

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def tolerance(dtype):
    return 64.0 * U + (HALF[dtype] + 2.0 ** -13 if dtype is not torch.float32 else 0.0)


def decay_of(kind, g):
    """(a, its slope)."""
    if kind == "sigmoid":
        return torch.sigmoid(g), torch.sigmoid(g) * torch.sigmoid(-g)
    return g.exp(), g.exp()


def rate_of(kind, b):
    if kind == "sigmoid":
        return torch.sigmoid(b), torch.sigmoid(b) * torch.sigmoid(-b)
    return b, torch.ones_like(b)


def delta_rule(q, k, v, gate, beta, h0, decay, rate, scale, dy=None, dlast=None):
    """One sequence: q, k [T, Hk, K], v [T, H, V], gate, beta [T, H], h0 [H, K, V], float64. (y, last) or, with dy,
    those and (dq, dk, dv, dgate, dbeta, dh0) and the sizes [T, H] that the errors of dgate and dbeta go by."""
    T, H = gate.shape
    Hk = q.shape[1]
    pick = torch.arange(H, device=v.device) // (H // Hk)
    a, da = decay_of(decay, gate)
    b, db = rate_of(rate, beta)
    qw, kw = q[:, pick], k[:, pick]
    states, y = [h0], torch.zeros_like(v)
    errors, pres = [], []
    for t in range(T):
        pre = a[t][:, None, None] * states[-1]
        e = v[t] - (pre * kw[t][:, :, None]).sum(1)
        states.append(pre + (b[t][:, None] * kw[t])[:, :, None] * e[:, None, :])
        pres.append(pre)
        errors.append(e)
        y[t] = scale * (states[-1] * qw[t][:, :, None]).sum(1)
    if dy is None:
        return y, states[-1]
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, dbeta = torch.zeros_like(gate), torch.zeros_like(beta)
    gate_size, rate_size = torch.zeros_like(gate), torch.zeros_like(gate)
    d = torch.zeros_like(h0) if dlast is None else dlast.clone()
    for t in range(T - 1, -1, -1):
        e, pre = errors[t], pres[t]
        dq[t].index_add_(0, pick, scale * (states[t + 1] * dy[t][:, None, :]).sum(2))
        d = d + scale * qw[t][:, :, None] * dy[t][:, None, :]
        through = (d * e[:, None, :]).sum(2)
        dbeta[t] = (through * kw[t]).sum(1) * db[t]
        rate_size[t] = (d * kw[t][:, :, None]).sum(1).norm(dim=1) * e.norm(dim=1) * db[t]
        gate_size[t] = d.norm(dim=(1, 2)) * states[t + 1].norm(dim=(1, 2))
        de = b[t][:, None] * (d * kw[t][:, :, None]).sum(1)
        dv[t] = de
        dk[t].index_add_(0, pick, b[t][:, None] * through - (pre * de[:, None, :]).sum(2))
        d = d - kw[t][:, :, None] * de[:, None, :]
        dg[t] = (d * states[t]).sum((1, 2)) * da[t]
        d = a[t][:, None, None] * d
    for t in range(0, T, 64):
        gate_size[t:t + 64] = gate_size[t:t + 64].norm(dim=0) * da[t:t + 64]
    return y, states[-1], dq, dk, dv, dg, dbeta, d, gate_size, rate_size


def qk_norm(x, w, kind, eps, freq, pos, pairs, dy=None):
    """x [rows, H, D], pos [rows], float64; y or (y, dx, dw, the sizes dx errs by), by automatic differentiation."""
    x = x.detach().requires_grad_(dy is not None)
    w = None if w is None else w.detach().requires_grad_(dy is not None)
    square = (x * x).mean(-1, keepdim=True) if kind == "rms" else (x * x).sum(-1, keepdim=True)
    z = x / torch.sqrt(square + eps)
    z = z * w if w is not None else z
    if freq is not None:
        n = freq.shape[0]
        f = (pos.double()[:, None] * freq)[:, None, :]
        c, s = torch.cos(f), torch.sin(f)
        i = torch.arange(n, device=x.device)
        i, j = (i, i + n) if pairs == "halves" else (2 * i, 2 * i + 1)
        y = z.clone()
        y[..., i], y[..., j] = z[..., i] * c - z[..., j] * s, z[..., j] * c + z[..., i] * s
    else:
        y = z
    if dy is None:
        return y
    grads = torch.autograd.grad(y, (x,) if w is None else (x, w), dy, retain_graph=True)
    # dx is the difference of the turned back dy w / n and its part along x: its error goes by the former
    dz, = torch.autograd.grad(y, z, dy)
    size = (dz if w is None else dz * w.detach()).abs() / torch.sqrt(square.detach() + eps)
    size = size.norm(dim=-1, keepdim=True).expand_as(dz) / dz.shape[-1] ** 0.5
    return y.detach(), grads[0], grads[1] if w is not None else None, size


def near(got, want, tol, what, rows=True, size_of=None):
    """Norms over the whole and, where the first axis is rows, over each row. size_of: what the error goes by, if not
    the result itself."""
    got, want = got.detach().double(), want.double()
    assert got.shape == want.shape, f"{what}: {tuple(got.shape)} for {tuple(want.shape)}"
    assert torch.isfinite(got).all(), f"{what}: not finite"
    if not got.numel():
        return
    by = want if size_of is None else torch.maximum(want.abs(), size_of)
    off, size = (got - want).norm(), by.norm()
    assert off <= tol * size + 1e-30, f"{what}: {float(off / size):.3g} off, {tol:.3g} allowed"
    if rows and got.shape[0] > 1:
        off, each = (t.reshape(t.shape[0], -1).norm(dim=1) for t in (got - want, by))
        most = 8.0 * tol * (each + size / got.shape[0] ** 0.5) + 1e-30
        worst = int((off / most).argmax())
        assert (off <= most).all(), f"{what}: row {worst} is {float(off[worst] / each[worst]):.3g} off its own norm"
