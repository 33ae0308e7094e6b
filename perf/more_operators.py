"""More sequence operators as measured cases: the gated delta rule (forward,
forward + backward, one serving step) and the norms of its queries and keys
with a position rotation (forward, forward + backward).

``run`` with ``own = False`` computes them in their plain form, in elementary
torch operations and 32 bits; with ``own = True`` it makes the package's
calls. ``exact`` computes them from their definitions in 64 bits.

  delta rule   per sequence and head, from S_{-1} = h0 (keys x values):
                 S_t = a_t S_{t-1} + b_t k_t (v_t - a_t S_{t-1}^T k_t)^T
                 y_t = scale S_t^T q_t
               a = sigmoid(gate) or exp(gate);  b = sigmoid(beta) or beta
  q/k norm     per head: y = R(position) (x w / n),  n = sqrt(sum x^2 + eps)
               or sqrt(mean x^2 + eps), R turning pairs of channels
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6
RUN = 64  # steps that the plain form takes together
TRAIN_MOST = 8 * 2048 * 16  # steps x heads of the largest listed training case
SCAN_MOST = 2 * TRAIN_MOST
STEP_MOST = 128 * 32 * 128 * 128  # state elements that the largest listed serving step touches
NORM_MOST = 16384 * 40 * 128  # elements of the largest listed norm


def listed():
    return [
        # one step of four streams, eight small heads on four of queries and keys: latency alone
        {"name": "delta step of 4 streams", "op": "step", "batch": 4, "key_heads": 4, "heads": 8, "dk": 64, "dv": 64,
         "dtype": "bf16", "decay": "sigmoid", "rate": "sigmoid"},
        # one step of a full serving batch: every stream's matrix states go through once
        {"name": "delta step of 128 streams", "op": "step", "batch": 128, "key_heads": 16, "heads": 32, "dk": 128,
         "dv": 128, "dtype": "bf16", "decay": "sigmoid", "rate": "sigmoid"},
        # a small operator's series (256 steps of 500 channels, 20 heads of 25) in FP32
        {"name": "delta small series", "op": "scan", "form": "batch", "batch": 1, "steps": 256, "key_heads": 20,
         "heads": 20, "dk": 25, "dv": 25, "dtype": "fp32", "decay": "exp", "rate": "value"},
        # prompts of unequal lengths packed one after the other, some of them empty
        {"name": "delta packed prompts", "op": "scan", "form": "packed", "batch": 45, "steps": 30011, "key_heads": 8,
         "heads": 16, "dk": 64, "dv": 128, "dtype": "fp16", "decay": "exp", "rate": "sigmoid"},
        # one very long series with few heads: little parallel work beside time
        {"name": "delta long series", "op": "scan", "form": "batch", "batch": 1, "steps": 65536, "key_heads": 8,
         "heads": 8, "dk": 128, "dv": 128, "dtype": "bf16", "decay": "sigmoid", "rate": "sigmoid"},
        # odd sizes: rows that start at any 2-byte address, ends inside every tile
        {"name": "delta odd sizes", "op": "scan", "form": "batch", "batch": 5, "steps": 1999, "key_heads": 7,
         "heads": 7, "dk": 75, "dv": 41, "dtype": "bf16", "decay": "sigmoid", "rate": "value"},
        # a training pass, eight series of 2048 steps with sixteen heads
        {"name": "delta training", "op": "scan_train", "form": "batch", "batch": 8, "steps": 2048, "key_heads": 16,
         "heads": 16, "dk": 128, "dv": 128, "dtype": "bf16", "decay": "sigmoid", "rate": "sigmoid"},
        # a padded training batch in FP32, one of its rows empty, heads that share queries and keys
        {"name": "delta training padded", "op": "scan_train", "form": "padded", "batch": 6, "steps": 1000,
         "key_heads": 2, "heads": 4, "dk": 64, "dv": 64, "dtype": "fp32", "decay": "sigmoid", "rate": "sigmoid"},
        # queries and keys of one step of four streams, far along their series
        {"name": "norm step of 4 streams", "op": "norm", "batch": 4, "steps": 1, "query_heads": 8, "key_heads": 8,
         "dim": 64, "rotated": 64, "pairs": "halves", "norm": "l2", "weight": False, "dtype": "bf16"},
        # a long prompt's, the larger heads of a model with shared keys
        {"name": "norm prompt", "op": "norm", "batch": 1, "steps": 16384, "query_heads": 32, "key_heads": 8,
         "dim": 128, "rotated": 128, "pairs": "halves", "norm": "rms", "weight": True, "dtype": "bf16"},
        # the training pass that goes with the delta rule's
        {"name": "norm training", "op": "norm_train", "batch": 8, "steps": 2048, "query_heads": 16, "key_heads": 16,
         "dim": 128, "rotated": 128, "pairs": "neighbours", "norm": "rms", "weight": True, "dtype": "bf16"},
        # odd head sizes in FP32, a part of each head rotated
        {"name": "norm training odd sizes", "op": "norm_train", "batch": 5, "steps": 1999, "query_heads": 7,
         "key_heads": 3, "dim": 75, "rotated": 50, "pairs": "halves", "norm": "l2", "weight": True, "dtype": "fp32"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "scan", "scan", "scan_train", "norm", "norm_train"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
    if op.startswith("norm"):
        case["dim"] = rng.choice([_log(rng, 8, 256), 64, 128])
        case["query_heads"], case["key_heads"] = _log(rng, 1, 64), _log(rng, 1, 32)
        each = case["dim"] * (case["query_heads"] + case["key_heads"])
        most = NORM_MOST * 2 // SIZES[case["dtype"]] // (3 if op == "norm_train" else 1)
        case["batch"] = _log(rng, 1, 64)
        case["steps"] = _log(rng, 1, max(1, min(16384, most // (each * case["batch"]))))
        case["rotated"] = rng.choice([0, case["dim"] // 4 * 2, case["dim"] // 2 * 2])
        case["pairs"] = rng.choice(["halves", "neighbours"])
        case["norm"] = rng.choice(["l2", "rms"])
        case["weight"] = rng.choice([True, False])
        return case
    case["decay"], case["rate"] = rng.choice(["sigmoid", "exp"]), rng.choice(["sigmoid", "value"])
    case["dk"], case["dv"] = (rng.choice([_log(rng, 8, 128), 64, 128]) for _ in range(2))
    case["key_heads"] = _log(rng, 1, 32)
    case["heads"] = case["key_heads"] * rng.choice([1, 1, 2, 4])
    if op == "step":
        case["batch"] = _log(rng, 1, max(1, min(256, STEP_MOST // (case["heads"] * case["dk"] * case["dv"]))))
        return case
    most = (TRAIN_MOST if op == "scan_train" else SCAN_MOST) * 2 // SIZES[case["dtype"]] // case["heads"]
    case["form"] = rng.choice(["batch", "padded", "packed"])
    case["steps"] = _log(rng, 1, min(65536, most))
    each = (case["steps"] + RUN - 1) // RUN  # runs of a sequence: short ones cost as much as a whole one
    room = most // RUN - each if case["form"] == "packed" else most // RUN // each
    case["batch"] = _log(rng, 1, max(1, min(128, room)))
    return case


def _held(case):
    """Steps that a batch holds on average."""
    if case["form"] == "packed":
        return case["steps"]
    return case["steps"] * case["batch"] * (0.5 if case["form"] == "padded" else 1.0)


def work(case):
    es, op = SIZES[case["dtype"]], case["op"]
    if op.startswith("norm"):
        rows = case["batch"] * case["steps"]
        n = rows * case["dim"] * (case["query_heads"] + case["key_heads"])
        params = 8 * case["dim"] if case["weight"] else 0
        if op == "norm":  # in, out; positions
            return {"bytes": 2 * es * n + 4 * rows + params, "flops": 8 * n}
        # x, dy in; y, dx out; gradients of the weights
        return {"bytes": 4 * es * n + 4 * rows + 2 * params, "flops": 28 * n}
    H, Hk, dk, dv = case["heads"], case["key_heads"], case["dk"], case["dv"]
    row = es * (2 * Hk * dk + H * dv + 2 * H)  # q, k, v, gate, beta of a step
    if op == "step":  # those in, y out; a state in and out
        return {"bytes": case["batch"] * (row + es * H * dv + 8 * H * dk * dv), "flops": 6 * case["batch"] * H * dk * dv}
    live, ends = _held(case), 4 * case["batch"] * H * dk * dv
    rows = case["steps"] * (1 if case["form"] == "packed" else case["batch"])
    if op == "scan":  # inputs, h0 in; y, last state out
        return {"bytes": live * row + rows * es * H * dv + 2 * ends, "flops": 6 * live * H * dk * dv}
    # inputs, dy, h0, dlast in; y, last state, gradients of every input, dh0 out
    return {"bytes": live * (row + es * H * dv) + rows * (row + es * H * dv) + 4 * ends,
            "flops": 20 * live * H * dk * dv}


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _lengths(gen, n, most):
    """Between nothing and all of a row; where there are several, one empty and one full."""
    t = torch.randint(0, most + 1, (n,), generator=gen, device="cuda", dtype=torch.int32)
    if n > 1:
        t[0], t[1] = 0, most
    return t


def _offsets(gen, n, total):
    """Cuts of a packed axis into n sequences, in order; equal cuts leave empty ones."""
    cuts = torch.randint(0, total + 1, (n + 1,), generator=gen, device="cuda", dtype=torch.int32)
    cuts[0], cuts[n] = 0, total
    if n > 2:
        cuts[1] = cuts[2]
    return torch.sort(cuts).values.to(torch.int32)


def _unit(t):
    return t * torch.rsqrt((t * t).sum(-1, keepdim=True) + EPS)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype, op = DTYPES[case["dtype"]], case["op"]
    s = {"case": case}
    if op.startswith("norm"):
        n, T, Hq, Hk, D = (case[w] for w in ("batch", "steps", "query_heads", "key_heads", "dim"))
        both = (_normal(gen, n, T, (Hq + Hk) * D) * (0.5 + torch.rand(((Hq + Hk) * D,), generator=gen, device="cuda"))).to(dtype)
        s["q"], s["k"] = both[..., :Hq * D].unflatten(-1, (Hq, D)), both[..., Hq * D:].unflatten(-1, (Hk, D))
        s["wq"] = 1.0 + 0.2 * _normal(gen, D) if case["weight"] else None
        s["wk"] = 1.0 + 0.2 * _normal(gen, D) if case["weight"] else None
        s["freq"] = None
        if case["rotated"]:
            at = torch.arange(case["rotated"] // 2, dtype=torch.float64, device="cuda")
            s["freq"] = 10000.0 ** (-2.0 * at / case["rotated"])
        # each series goes on from where it stands, up to half a million steps along
        start = torch.randint(0, 500_000, (n, 1), generator=gen, device="cuda", dtype=torch.int32)
        s["pos"] = start + torch.arange(T, dtype=torch.int32, device="cuda")
        if op == "norm_train":
            s["dq"], s["dk"] = _normal(gen, n, T, Hq, D).to(dtype), _normal(gen, n, T, Hk, D).to(dtype)
        return s
    n, H, Hk, dk, dv = (case[w] for w in ("batch", "heads", "key_heads", "dk", "dv"))
    rows = (n,) if op == "step" else (case["steps"],) if case["form"] == "packed" else (n, case["steps"])
    s["q"], s["k"] = (_unit(_normal(gen, *rows, Hk, dk)).to(dtype) for _ in range(2))
    # values, gates and rates are parts of one projection, as a layer has them
    p = torch.empty(rows + (H * (dv + 2),), dtype=dtype, device="cuda")
    s["v"], s["gate"], s["beta"] = p[..., :H * dv].unflatten(-1, (H, dv)), p[..., H * dv:H * (dv + 1)], p[..., H * (dv + 1):]
    s["v"].copy_(_normal(gen, *rows, H, dv))
    # memories from a few steps to some hundreds, by head
    g = _normal(gen, *rows, H) + 2.0 + 4.0 * torch.rand((H,), generator=gen, device="cuda")
    s["gate"].copy_(g if case["decay"] == "sigmoid" else torch.nn.functional.logsigmoid(g))
    r = _normal(gen, *rows, H)
    s["beta"].copy_(r if case["rate"] == "sigmoid" else torch.sigmoid(r))
    s["scale"] = dk ** -0.5
    if op == "step":
        places = n + n // 2 + 1  # a state cache with more places than streams
        s["state"] = 0.3 * _normal(gen, places, H, dk, dv)
        s["slots"] = torch.randperm(places, generator=gen, device="cuda")[:n].to(torch.int32)
        if n > 8:
            s["slots"][3] = -1  # an idle place in the batch
        return s
    T = case["steps"]
    s["h0"] = 0.3 * _normal(gen, n, H, dk, dv)
    s["lengths"] = _lengths(gen, n, T) if case["form"] == "padded" else None
    s["offsets"] = _offsets(gen, n, T) if case["form"] == "packed" else None
    if op == "scan_train":
        s["dy"] = _normal(gen, *rows, H, dv).to(dtype)
        s["dlast"] = 0.3 * _normal(gen, n, H, dk, dv)
    return s


# ------------------------------------------------------------- plain forms
def _runs(case, s):
    """The steps in runs of RUN that no sequence's end cuts: rows [runs, RUN] of the flat axis and which of them are
    held, each run's sequence, whether it is that one's first, and each sequence's last run (or -1)."""
    n, T = case["batch"], case["steps"]
    dev, at = "cuda", torch.arange(RUN, device="cuda")
    if case["form"] == "packed":
        o = s["offsets"].long()
        base, count = o[:-1], o[1:] - o[:-1]
    else:
        base = torch.arange(n, device=dev) * T
        count = s["lengths"].long() if case["form"] == "padded" else torch.full((n,), T, device=dev)
    each = (count + RUN - 1) // RUN
    ends = torch.cumsum(each, 0)
    runs = T // RUN + n if case["form"] == "packed" else n * ((T + RUN - 1) // RUN)
    i = torch.arange(runs, device=dev)
    seq = (i[:, None] >= ends[None, :]).sum(1).clamp(max=n - 1)
    place = i - (ends - each)[seq]  # the run's number in its sequence; those behind the last one hold nothing
    step = place[:, None] * RUN + at
    held = (step < count[seq][:, None]) & (i < ends[-1])[:, None]
    rows = torch.where(held, base[seq][:, None] + step, 0)
    return rows, held, seq, (place == 0) | (i >= ends[-1]), torch.where(each > 0, ends - 1, -1)


def _lower_inverse(a):
    """(1 + a)^-1 of strictly lower triangular a, from blocks of one row to the whole by doubling."""
    lead, n, d = a.shape[:-2], a.shape[-1], 1
    t = torch.ones(lead + (n, 1, 1), device=a.device)
    while d < n:
        m = n // (2 * d)
        low = a.reshape(lead + (m, 2 * d, m, 2 * d)).diagonal(dim1=-4, dim2=-2).movedim(-1, -3)[..., d:, :d]
        t = t.reshape(lead + (m, 2, d, d))
        first, second = t[..., 0, :, :], t[..., 1, :, :]
        left = torch.cat([first, -(second @ (low @ first))], -2)
        right = torch.cat([torch.zeros_like(first), second], -2)
        t, d = torch.cat([left, right], -1), 2 * d
    return t.reshape(a.shape)


def _plain_delta(case, s, q, k, v, gate, beta, h0):
    """(y, last state) in 32 bits from inputs in 32 bits; runs of steps at once, their maps joined by doubling."""
    n, H, Hk, dk, dv = (case[w] for w in ("batch", "heads", "key_heads", "dk", "dv"))
    rows, held, seq, first, last = _runs(case, s)

    def pick(t, heads):  # [runs, heads, RUN, ...]
        t = t.reshape((-1,) + t.shape[-(t.dim() - len(s["gate"].shape) + 1):])
        t = torch.where(held.reshape(held.shape + (1,) * (t.dim() - 1)), t[rows], 0.0).transpose(1, 2)
        return t.repeat_interleave(H // heads, 1) if heads < H else t

    q, k, v, g, b = pick(q, Hk), pick(k, Hk), pick(v, H), pick(gate, H), pick(beta, H)
    on = held[:, None, :]
    if case["decay"] == "sigmoid":
        g = torch.nn.functional.logsigmoid(g)
    if case["rate"] == "sigmoid":
        b = torch.sigmoid(b)
    g, b = torch.where(on, g, 0.0), torch.where(on, b, 0.0)
    total = torch.cumsum(g.double(), -1)
    lower = torch.ones(RUN, RUN, device="cuda", dtype=torch.bool).tril()
    between = torch.exp(torch.where(lower, total[..., :, None] - total[..., None, :], -1e4).float())
    into, out = torch.exp(total.float())[..., None], torch.exp((total[..., -1:] - total).float())[..., None]
    kT = k.transpose(-1, -2)
    t = _lower_inverse(((k @ kT) * between * b[..., None]).tril(-1))
    w, u = t @ (b[..., None] * into * k), t @ (b[..., None] * v)
    kout = (out * k).transpose(-1, -2)
    m = into[..., -1:, :] * torch.eye(dk, device="cuda") - kout @ w
    x = kout @ u
    start = first[:, None, None, None]
    x = x + torch.where(start, m @ h0[seq], 0.0)
    m, d = torch.where(start, 0.0, m), 1
    while d < (case["steps"] + RUN - 1) // RUN:
        x = torch.cat([x[:d], x[d:] + m[d:] @ x[:-d]])
        m = torch.cat([m[:d], m[d:] @ m[:-d]])
        d *= 2
    before = torch.where(start, h0[seq], torch.cat([x[:1], x[:-1]]))
    u = u - w @ before
    y = s["scale"] * (into * (q @ before) + ((q @ kT) * between) @ u)
    flat = torch.zeros((s["gate"].numel() // H + 1, H, dv), device="cuda")
    y = flat.index_put((torch.where(held, rows, flat.shape[0] - 1),), torch.where(on[..., None], y, 0.0).transpose(1, 2))
    return y[:-1].reshape(s["v"].shape), torch.where((last >= 0)[:, None, None, None], x[last.clamp(min=0)], h0)


def _plain_scan(case, s, train):
    dtype = s["q"].dtype
    names = ("q", "k", "v", "gate", "beta", "h0")
    # copies of its own for each input, gradients or not
    leaves = [s[w].float().clone().requires_grad_(train) for w in names]
    y, last = _plain_delta(case, s, *leaves)
    if not train:
        return y.to(dtype), last
    grads = torch.autograd.grad((y, last), leaves, (s["dy"].float(), s["dlast"]))
    return (y.detach().to(dtype), last.detach()) + tuple(t.to(s[w].dtype) for t, w in zip(grads, names))


def _plain_step(case, s):
    n, H, Hk = case["batch"], case["heads"], case["key_heads"]
    q, k = (s[w].float().repeat_interleave(H // Hk, 1) for w in "qk")
    v, g, b = s["v"].float(), s["gate"].float(), s["beta"].float()
    a = (torch.sigmoid(g) if case["decay"] == "sigmoid" else torch.exp(g))[..., None]
    b = (torch.sigmoid(b) if case["rate"] == "sigmoid" else b)[..., None]
    on = s["slots"] >= 0
    at = s["slots"].long().clamp(min=0)
    h = s["state"][at] * a[..., None]
    e = v - (k[..., None, :] @ h)[..., 0, :]
    h = h + (b * k)[..., :, None] * e[..., None, :]
    y = torch.where(on[:, None, None], s["scale"] * (q[..., None, :] @ h)[..., 0, :], 0.0)
    keep = torch.where(on[:, None, None, None], h, s["state"][at])
    # an idle stream writes over no other's place: it has a row of its own behind the cache
    wide = torch.cat([s["state"], s["state"][:1]])
    wide[torch.where(on, at, s["state"].shape[0])] = keep
    s["state"].copy_(wide[:-1])
    return y.to(s["v"].dtype), s["state"]


def _turns(case, s):
    """(cos, sin) [batch, steps, 1, pairs] of the angles, taken in 64 bits."""
    angle = s["pos"].double()[..., None, None] * s["freq"]
    return torch.cos(angle).float(), torch.sin(angle).float()


def _rotate(case, x, c, sn):
    R = case["rotated"]
    if case["pairs"] == "halves":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        return torch.cat([a * c - b * sn, b * c + a * sn, x[..., R:]], -1)
    a, b = x[..., 0:R:2], x[..., 1:R:2]
    return torch.cat([torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2), x[..., R:]], -1)


def _plain_norm(case, s, train):
    out, grads = [], []
    c, sn = _turns(case, s) if s["freq"] is not None else (None, None)
    for x, w, dy in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
        dtype, x = x.dtype, x.float()
        count = x.shape[-1] if case["norm"] == "rms" else 1
        r = torch.rsqrt((x * x).sum(-1, keepdim=True) / count + EPS)
        xhat = x * r
        y = xhat * w if w is not None else xhat
        out.append((_rotate(case, y, c, sn) if c is not None else y).to(dtype))
        if train:
            dz = dy.float()
            dz = _rotate(case, dz, c, -sn) if c is not None else dz  # the turn back
            t = dz * w if w is not None else dz
            grads.append((r * (t - xhat * ((t * xhat).sum(-1, keepdim=True) / count))).to(dtype))
            grads.append((dz * xhat).sum((0, 1, 2)) if w is not None else None)
    return tuple(out) + tuple(g for g in grads if g is not None)


def run(s):
    case = s["case"]
    op = case["op"]
    train = op.endswith("train")
    if not own:
        if op == "step":
            return _plain_step(case, s)
        return _plain_scan(case, s, train) if op.startswith("scan") else _plain_norm(case, s, train)
    import fft_block_toeplitz_amd as fm

    if op.startswith("norm"):
        how = {"norm": case["norm"], "eps": EPS, "frequencies": s["freq"], "positions": s["pos"], "pairs": case["pairs"]}
        out = fm.qk_norm(s["q"], s["k"], s["wq"], s["wk"], **how)
        if train:
            dq, dk, dwq, dwk = fm.qk_norm_backward(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], **how)
            out = out + ((dq, dwq, dk, dwk) if case["weight"] else (dq, dk))
        return out
    how = {"decay": case["decay"], "rate": case["rate"], "scale": s["scale"]}
    inputs = s["q"], s["k"], s["v"], s["gate"], s["beta"]
    if op == "step":
        return fm.delta_rule_step(*inputs, s["state"], s["slots"], **how), s["state"]
    how.update(lengths=s["lengths"], offsets=s["offsets"])
    if not train:
        return fm.delta_rule(*inputs, s["h0"], **how)
    y, last, carries = fm.delta_rule(*inputs, s["h0"], save=True, **how)
    return (y, last) + fm.delta_rule_backward(s["dy"], *inputs, carries, s["h0"], s["dlast"], **how)


# ------------------------------------------------------------ in 64 bits
def _exact_decay(case, g):
    """The decay and its slope."""
    if case["decay"] == "sigmoid":
        a = 1.0 / (1.0 + torch.exp(-g))
        return a, a / (1.0 + torch.exp(g))
    return g.exp(), g.exp()


def _exact_rate(case, b):
    if case["rate"] == "sigmoid":
        r = 1.0 / (1.0 + torch.exp(-b))
        return r, r / (1.0 + torch.exp(b))
    return b, torch.ones_like(b)


def _times(h, x):
    """h^T x for matrices [keys, values] and vectors of keys."""
    return (x.unsqueeze(-2) @ h).squeeze(-2)


def _exact_scan(case, s, train):
    """The definition step by step; a sequence is a row of a padded batch, and where it has ended its state stays."""
    n, H, Hk, dk, dv = (case[w] for w in ("batch", "heads", "key_heads", "dk", "dv"))
    packed = case["form"] == "packed"
    spans = [(0, case["steps"])] * n
    if case["form"] == "padded":
        spans = [(0, m) for m in s["lengths"].tolist()]
    elif packed:
        o = s["offsets"].tolist()
        spans = list(zip(o[:-1], o[1:]))
    longest = max(e - b for b, e in spans)
    seconds = longest * (30 if train else 8) * (1.2e-5 + n * H * dk * dv * 1.5e-11)
    state = n * H * dk * dv * 8
    part = max(1, min(64, int(16e9 // state)))  # steps whose states are kept at once
    if seconds > 12.0 or state * (longest // part + 1) > 48e9 or longest * n * H * (3 * dk + 3 * dv) * 8 > 40e9:
        return None

    def rows(t):  # [longest, n, ...] in 64 bits
        if case["form"] == "batch":
            return t.transpose(0, 1).double()
        p = torch.zeros((longest, n) + tuple(t.shape[-(t.dim() - (1 if packed else 2)):]), dtype=torch.float64, device="cuda")
        for i, (b, e) in enumerate(spans):
            p[:e - b, i] = t[b:e] if packed else t[i, :e]
        return p

    def back(p, like):
        t = torch.zeros(like.shape, dtype=torch.float64, device="cuda")
        for i, (b, e) in enumerate(spans):
            if packed:
                t[b:e] = p[:e - b, i]
            else:
                t[i, :e] = p[:e, i]
        return t

    q, k, v = rows(s["q"]), rows(s["k"]), rows(s["v"])
    wide = [h // (H // Hk) for h in range(H)]  # the head of queries and keys of each head
    on = torch.tensor([[float(t < e - b) for b, e in spans] for t in range(longest)], dtype=torch.float64)
    on = on.cuda().reshape(longest, n, 1)
    a, da = _exact_decay(case, rows(s["gate"]))
    r, dr = _exact_rate(case, rows(s["beta"]))
    a, r = a * on + (1.0 - on), r * on
    scale = s["scale"]

    def step(t, h):
        kt, pre = k[t][:, wide], a[t][..., None, None] * h
        e = v[t] - _times(pre, kt)
        return pre, e, pre + (r[t][..., None] * kt)[..., :, None] * e[..., None, :]

    y = torch.zeros((longest, n, H, dv), dtype=torch.float64, device="cuda")
    h, kept = s["h0"].double(), []
    for t in range(longest):
        if train and t % part == 0:
            kept.append(h)
        h = step(t, h)[2]
        y[t] = scale * _times(h, q[t][:, wide]) * on[t][..., None]
    out = back(y, s["v"]), h
    if not train:
        return out
    dy = rows(s["dy"]) * on[..., None]
    dq, dkk, dvv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(a), torch.zeros_like(r)
    d = s["dlast"].double()

    def joined(x):  # the gradients of heads that share queries and keys
        return x.reshape(n, Hk, H // Hk, dk).sum(2)

    for c in range(len(kept) - 1, -1, -1):
        states = [kept[c]]
        for t in range(c * part, min(longest, (c + 1) * part) - 1):
            states.append(step(t, states[-1])[2])
        for t in range(min(longest, (c + 1) * part) - 1, c * part - 1, -1):
            h = states[t - c * part]
            pre, e, after = step(t, h)
            kt, qt, rt = k[t][:, wide], q[t][:, wide], r[t][..., None]
            dq[t] = joined(scale * (after @ dy[t][..., None]).squeeze(-1))
            d = d + scale * qt[..., :, None] * dy[t][..., None, :]
            through = (d @ e[..., None]).squeeze(-1)
            db[t] = (kt * through).sum(-1)
            de = rt * _times(d, kt)
            dvv[t] = de
            dkk[t] = joined(rt * through - (pre @ de[..., None]).squeeze(-1))
            d = d - kt[..., :, None] * de[..., None, :]
            dg[t] = (d * h).sum((-1, -2))
            d = a[t][..., None, None] * d
    return out + (back(dq, s["q"]), back(dkk * on[..., None], s["k"]), back(dvv, s["v"]), back(dg * da * on, s["gate"]),
                  back(db * dr * on, s["beta"]), d)


def _exact_step(case, s):
    H, Hk = case["heads"], case["key_heads"]
    state = s["state"].double()
    y = torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
    a, r = _exact_decay(case, s["gate"].double())[0], _exact_rate(case, s["beta"].double())[0]
    wide = [h // (H // Hk) for h in range(H)]
    q, k, v = s["q"].double()[:, wide], s["k"].double()[:, wide], s["v"].double()
    for i, place in enumerate(s["slots"].tolist()):
        if place >= 0:
            pre = a[i][:, None, None] * state[place]
            e = v[i] - _times(pre, k[i])
            state[place] = pre + (r[i][:, None] * k[i])[:, :, None] * e[:, None, :]
            y[i] = s["scale"] * _times(state[place], q[i])
    return y, state


def _exact_norm(case, s, train):
    """The definition, pairs as complex numbers; the gradients by automatic differentiation in 64 bits."""
    R, out, grads = case["rotated"], [], []
    for x, w, dy in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
        x = x.double().detach().requires_grad_(train)
        w = None if w is None else w.double().requires_grad_(train)
        square = x.square()
        size = torch.sqrt((square.mean(-1) if case["norm"] == "rms" else square.sum(-1)) + EPS)
        y = x / size.unsqueeze(-1)
        if w is not None:
            y = y * w
        if R:
            turn = torch.polar(torch.ones_like(s["freq"]), s["pos"].double().unsqueeze(-1) * s["freq"]).unsqueeze(-2)
            if case["pairs"] == "halves":
                z = torch.complex(y[..., :R // 2], y[..., R // 2:R]) * turn
                y = torch.cat([z.real, z.imag, y[..., R:]], -1)
            else:
                z = torch.complex(y[..., 0:R:2], y[..., 1:R:2]) * turn
                y = torch.cat([torch.view_as_real(z).flatten(-2), y[..., R:]], -1)
        out.append(y.detach())
        if train:
            grads += torch.autograd.grad(y, (x,) if w is None else (x, w), dy.double())
    return tuple(out) + tuple(grads)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "step":
        return _exact_step(case, s)
    return _exact_scan(case, s, op.endswith("train")) if op.startswith("scan") else _exact_norm(case, s, op.endswith("train"))
