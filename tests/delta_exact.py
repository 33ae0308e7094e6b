"""The gradients of the gated delta rule for each head by itself, step by step in float64, and how far sums in float32 may
leave the gates' gradients off.

The kernels take the gradient of log a_t as the sum, over the steps i >= t of a run of 64, of what each step's decay is a
factor of: inner products over the keys of q_i with dq_i and of k_i with the two parts of dk_i, and at the run's end the
product of the state with its gradient. A term of such an inner product comes from sums over up to 128 keys or 64 values
at a time and over the run's steps, some 400 roundings in line of 2^-24 of either sign, so it is off by sqrt(400) = 20 of
2^-24 of itself, whatever the sums cancel: the errors' size is the root of the sum of the squares of all terms,

    size_t = (sum_{i >= t} |q_i o dq_i|^2 + |k_i o b d e|^2 + |k_i o S de|^2 + |S_end o D_end|^2)^(1/2),  o by elements,

and 20 * 2^-24 * size_t times the slope of log a (1 - a, or 1) is what an error is on average. Three times that is allowed in the mean square over a
head's steps, and 24 times (8 standard deviations of the former) for each step. On top of it, the result's own type
rounds by half a step."""
import torch

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# the smallest number that rounds to within half a step of itself; below it, half of its step
SMALL = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def decay_of(kind, g):
    return (torch.sigmoid(g), torch.sigmoid(g) * torch.sigmoid(-g)) if kind == "sigmoid" else (g.exp(), g.exp())


def rate_of(kind, b):
    return (torch.sigmoid(b), torch.sigmoid(b) * torch.sigmoid(-b)) if kind == "sigmoid" else (b, torch.ones_like(b))


def gradients(q, k, v, gate, beta, h0, decay, rate, scale, dy, dlast):
    """One sequence in float64: q, k [T, Hk, K], v, dy [T, H, V], gate, beta [T, H], h0, dlast [H, K, V]. A dict of y,
    last, dq, dk (summed over the heads that share them), dv, dgate, dbeta, dh0, and size [T, H], times log a's slope."""
    T, H = gate.shape
    Hk, K = q.shape[1:]
    pick = torch.arange(H, device=v.device) // (H // Hk)
    a, slope = decay_of(decay, gate)
    b, turn = rate_of(rate, beta)
    qw, kw = q[:, pick], k[:, pick]
    states, pres, errors, y = [h0], [], [], torch.zeros_like(v)
    for t in range(T):
        pre = a[t][:, None, None] * states[-1]
        e = v[t] - (pre * kw[t][:, :, None]).sum(1)
        states.append(pre + (b[t][:, None] * kw[t])[:, :, None] * e[:, None, :])
        pres.append(pre)
        errors.append(e)
        y[t] = scale * (states[-1] * qw[t][:, :, None]).sum(1)
    dq, dk = torch.zeros_like(qw), torch.zeros_like(kw)
    dv, dgate, dbeta, size = torch.zeros_like(v), torch.zeros_like(gate), torch.zeros_like(beta), torch.zeros_like(gate)
    d, squares = dlast.clone(), None
    for t in range(T - 1, -1, -1):
        if t == T - 1 or t % 64 == 63:
            squares = ((states[t + 1] * d) ** 2).sum((1, 2))
        dq[t] = scale * (states[t + 1] * dy[t][:, None, :]).sum(2)
        d = d + scale * qw[t][:, :, None] * dy[t][:, None, :]
        through = (d * errors[t][:, None, :]).sum(2)
        dbeta[t] = (through * kw[t]).sum(1) * turn[t]
        de = b[t][:, None] * (d * kw[t][:, :, None]).sum(1)
        dv[t] = de
        there, found = b[t][:, None] * through, (pres[t] * de[:, None, :]).sum(2)
        dk[t] = there - found
        d = d - kw[t][:, :, None] * de[:, None, :]
        dgate[t] = (d * states[t]).sum((1, 2)) * slope[t]
        d = a[t][:, None, None] * d
        squares = squares + ((qw[t] * dq[t]) ** 2 + (kw[t] * there) ** 2 + (kw[t] * found) ** 2).sum(1)
        size[t] = squares.sqrt() * (1.0 - a[t] if decay == "sigmoid" else 1.0)
    share = lambda x: x.unflatten(1, (Hk, H // Hk)).sum(2)  # noqa: E731
    return {"y": y, "last": states[-1], "dq": share(dq), "dk": share(dk), "dv": dv, "dgate": dgate, "dbeta": dbeta,
            "dh0": d, "size": size}


def gates_off(got, want, size, dtype):
    """What is wrong with a head's gradients of its gate [T], or None."""
    got, want = got.detach().double(), want.double()
    if not torch.isfinite(got).all():
        return "not finite"
    off = (got - want).abs()
    stored = HALF[dtype] * want.abs() + SMALL[dtype]
    # what a store's rounding does not explain, in units of the sums' errors
    sums = (off - stored).clamp(min=0.0) / (20 * U * size + 1e-300)
    if not (sums <= 24).all():
        t = int(sums.argmax())
        return f"step {t}: {float(off[t]):.3g} off {float(want[t]):.3g}, the sums' error {float(sums[t]):.3g} times over"
    mean = float(sums.square().mean().sqrt())
    if not mean <= 3:
        return f"the sums' error {mean:.3g} times over in the mean square"
    return None
