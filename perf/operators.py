"""The sequence operators as measured cases: a gated linear recurrence along
time (forward, forward + backward, one serving step) and group normalisation
with an activation over channels-last fields (forward, forward + backward).

``run`` with ``own = False`` computes them in their plain form, in elementary
torch operations and 32 bits; with ``own = True`` it makes the package's
calls. ``exact`` computes them from their definitions in 64 bits.

  recurrence   h_t = a_t h_{t-1} + u_t per channel, from h_{-1} = h0;
               a = sigmoid(g), exp(g) or g;  u = x or (1 - a) x
  group norm   y = act((x - mean) / sqrt(var + eps) * w + b), mean and
               variance over a sample's rows and one group of channels
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5
LARGEST = 80_000_000  # elements of the largest listed case (training)


def listed():
    return [
        # one step of a stream that answers four requests, at a small operator's 500 channels: latency alone
        {"name": "step of 4 requests", "op": "step", "batch": 4, "channels": 500, "dtype": "bf16",
         "decay": "sigmoid", "drive": "complement"},
        # one step of a full serving batch at 5000 channels, a few of its places idle
        {"name": "step of 512 requests", "op": "step", "batch": 512, "channels": 5000, "dtype": "bf16",
         "decay": "sigmoid", "drive": "complement"},
        # a small operator's whole series (256 steps of 500 channels) in FP32
        {"name": "scan small series", "op": "scan", "form": "batch", "batch": 1, "steps": 256, "channels": 500,
         "dtype": "fp32", "decay": "value", "drive": "plain"},
        # prompts of unequal lengths packed one after the other, some of them empty
        {"name": "scan packed prompts", "op": "scan", "form": "packed", "batch": 45, "steps": 30011,
         "channels": 2048, "dtype": "fp16", "decay": "exp", "drive": "plain"},
        # one very long series: little parallel work across channels
        {"name": "scan long series", "op": "scan", "form": "batch", "batch": 1, "steps": 65536, "channels": 1024,
         "dtype": "bf16", "decay": "sigmoid", "drive": "complement"},
        # odd sizes, rows that start at any 2-byte address
        {"name": "scan odd sizes", "op": "scan", "form": "batch", "batch": 5, "steps": 1999, "channels": 1001,
         "dtype": "bf16", "decay": "sigmoid", "drive": "plain"},
        # a training pass at 5000 channels and 2000 steps, eight series
        {"name": "scan training", "op": "scan_train", "form": "batch", "batch": 8, "steps": 2000, "channels": 5000,
         "dtype": "bf16", "decay": "sigmoid", "drive": "complement"},
        # a padded training batch in FP32, one of its rows empty
        {"name": "scan training padded", "op": "scan_train", "form": "padded", "batch": 6, "steps": 1000,
         "channels": 500, "dtype": "fp32", "decay": "sigmoid", "drive": "complement"},
        # the normalisation behind the small step: single tokens, odd groups
        {"name": "norm of 4 tokens", "op": "norm", "form": "tokens", "batch": 4, "rows": 1, "groups": 20,
         "width": 25, "dtype": "bf16", "activation": "silu"},
        # a field of 64 x 64 points, channels last, inference
        {"name": "norm field", "op": "norm", "form": "field", "batch": 4, "rows": 4096, "groups": 32, "width": 16,
         "dtype": "bf16", "activation": "silu"},
        # the training pass that goes with the recurrence's: every token by itself
        {"name": "norm training tokens", "op": "norm_train", "form": "tokens", "batch": 16000, "rows": 1,
         "groups": 25, "width": 200, "dtype": "bf16", "activation": "silu"},
        # large fields in FP16, groups of ten channels
        {"name": "norm training fields", "op": "norm_train", "form": "field", "batch": 2, "rows": 16384,
         "groups": 32, "width": 10, "dtype": "fp16", "activation": "gelu"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "scan", "scan", "scan_train", "norm", "norm_train"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
    most = LARGEST * 2 // SIZES[case["dtype"]] // (1 if op.endswith("train") else 2)
    if op in ("step", "scan", "scan_train"):
        case["decay"] = rng.choice(["sigmoid", "sigmoid", "exp", "value"])
        case["drive"] = rng.choice(["complement", "plain"])
        case["channels"] = _log(rng, 24, 8192)
        if op == "step":
            case["batch"] = _log(rng, 1, 1024)
            return case
        case["form"] = rng.choice(["batch", "padded", "packed"])
        case["steps"] = _log(rng, 1, 65536)
        if case["form"] == "packed":  # steps: of all sequences together
            case["steps"] = max(1, min(case["steps"], most // case["channels"]))
            case["batch"] = _log(rng, 1, 256)
        else:
            case["steps"] = max(1, min(case["steps"], most // case["channels"]))
            case["batch"] = _log(rng, 1, max(1, min(256, most // (case["steps"] * case["channels"]))))
        return case
    case["activation"] = rng.choice(["none", "silu", "gelu"])
    case["form"] = rng.choice(["tokens", "field", "padded"])
    case["groups"] = _log(rng, 1, 64)
    case["width"] = _log(rng, 1, max(1, 8192 // case["groups"]))
    channels = case["groups"] * case["width"]
    if case["form"] == "tokens":
        case["rows"] = 1
        case["batch"] = _log(rng, 1, max(1, min(65536, most // channels)))
    else:
        case["rows"] = _log(rng, 2, max(2, min(65536, most // channels)))
        case["batch"] = _log(rng, 1, max(1, min(64, most // (channels * case["rows"]))))
    return case


def _live(case):
    """The share of rows that a padded batch holds on average."""
    return 0.5 if case["form"] == "padded" else 1.0


def work(case):
    es, op = SIZES[case["dtype"]], case["op"]
    if op == "step":  # x, gate and state in; h and state out
        n = case["batch"] * case["channels"]
        return {"bytes": n * (3 * es + 8), "flops": 10 * n}
    if op in ("scan", "scan_train"):
        C, rows = case["channels"], case["steps"] * (1 if case["form"] == "packed" else case["batch"])
        read, held = rows * _live(case) * C, rows * C
        ends = case["batch"] * C * 4
        if op == "scan":  # x, gate, h0 in; h, last state out
            return {"bytes": es * (2 * read + held) + 2 * ends, "flops": 10 * read}
        # x, gate, dh, h0, dlast in; h, last state, dx, dgate, dh0 out
        return {"bytes": es * (3 * read + 3 * held) + 4 * ends, "flops": 26 * read}
    C = case["groups"] * case["width"]
    held = case["batch"] * case["rows"] * C
    read = held * _live(case)
    if op == "norm":
        return {"bytes": es * (read + held) + 8 * C, "flops": 14 * read}
    return {"bytes": es * (2 * read + 2 * held) + 16 * C, "flops": 40 * read}


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


def _gates(gen, kind, shape):
    """Gate inputs: memories from a few steps to some hundreds, by channel."""
    by_channel = 1.0 + 4.0 * torch.rand((shape[-1],), generator=gen, device="cuda")
    g = _normal(gen, *shape).add_(by_channel)  # sigmoid(g): 0.3 .. 0.999
    if kind == "sigmoid":
        return g
    return torch.sigmoid(g) if kind == "value" else torch.nn.functional.logsigmoid(g)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype, op = DTYPES[case["dtype"]], case["op"]
    s = {"case": case}
    if op == "step":
        n, C = case["batch"], case["channels"]
        s["x"] = _normal(gen, n, C).to(dtype)
        s["gate"] = _gates(gen, case["decay"], (n, C)).to(dtype)
        s["state"] = 0.3 * _normal(gen, 2 * n, C)  # a state cache with twice the places
        s["slots"] = torch.randperm(2 * n, generator=gen, device="cuda")[:n].to(torch.int32)
        if n > 8:
            s["slots"][3] = -1  # an idle place in the batch
        return s
    if op in ("scan", "scan_train"):
        n, T, C = case["batch"], case["steps"], case["channels"]
        shape = (T, C) if case["form"] == "packed" else (n, T, C)
        # the two halves of one projection, as a layer has them
        both = torch.empty(shape[:-1] + (2 * C,), dtype=dtype, device="cuda")
        both[..., :C] = _normal(gen, *shape)
        both[..., C:] = _gates(gen, case["decay"], shape)
        s["x"], s["gate"] = both[..., :C], both[..., C:]
        s["h0"] = 0.3 * _normal(gen, n, C)
        s["lengths"] = _lengths(gen, n, T) if case["form"] == "padded" else None
        s["offsets"] = _offsets(gen, n, T) if case["form"] == "packed" else None
        if op == "scan_train":
            s["dh"] = _normal(gen, *shape).to(dtype)
            s["dlast"] = _normal(gen, n, C)
        return s
    n, S, G, C = case["batch"], case["rows"], case["groups"], case["groups"] * case["width"]
    shape = (n, C) if case["form"] == "tokens" else (n, S, C)
    s["x"] = (_normal(gen, *shape) * (0.5 + torch.rand((C,), generator=gen, device="cuda")) + _normal(gen, C)).to(dtype)
    s["weight"] = 1.0 + 0.2 * _normal(gen, C)
    s["bias"] = 0.2 * _normal(gen, C)
    s["lengths"] = _lengths(gen, n, S) if case["form"] == "padded" else None
    if op == "norm_train":
        s["dy"] = _normal(gen, *shape).to(dtype)
    return s


# ------------------------------------------------------------- plain forms
def _plain_terms(case, x, gate):
    """(a, u, da/dg) in 32 bits."""
    x, g = x.float(), gate.float()
    if case["decay"] == "sigmoid":
        a, rest = torch.sigmoid(g), torch.sigmoid(-g)
        slope = a * rest
    elif case["decay"] == "exp":
        a, rest = torch.exp(g), -torch.expm1(g)
        slope = a
    else:
        a, rest, slope = g, 1.0 - g, torch.ones_like(g)
    return a, rest, (rest * x if case["drive"] == "complement" else x), slope, x


def _plain_scan(a, u):
    """h_t = a_t h_{t-1} + u_t from zero along axis 1, by doubling the span that each step has joined."""
    a, u, d = a.clone(), u.clone(), 1
    while d < a.shape[1]:
        u[:, d:] = u[:, d:] + a[:, d:] * u[:, :-d]
        a[:, d:] = a[:, d:] * a[:, :-d]
        d *= 2
    return u


def _layout(case, s):
    """Rows of each sequence's first and last step on the (batch, steps) axes, which sequences hold any, and which steps are held."""
    n, T = case["batch"], case["steps"]
    at = torch.arange(n, device="cuda")
    if case["form"] == "packed":
        o = s["offsets"].long()
        first, last, some = o[:-1], o[1:] - 1, o[1:] > o[:-1]
        return torch.zeros_like(at), first, last, some, None
    if case["form"] == "padded":
        n_of = s["lengths"].long()
        held = torch.arange(T, device="cuda")[None, :] < n_of[:, None]
        return at, torch.zeros_like(at), n_of - 1, n_of > 0, held[..., None]
    return at, torch.zeros_like(at), torch.full_like(at, T - 1), torch.ones_like(at, dtype=torch.bool), None


def _plain_recurrence(case, s, train):
    dtype = s["x"].dtype
    x, gate = (s["x"][None], s["gate"][None]) if case["form"] == "packed" else (s["x"], s["gate"])
    b, first, last, some, held = _layout(case, s)
    a, rest, u, slope, x = _plain_terms(case, x, gate)
    if held is not None:
        a, u = torch.where(held, a, 0.0), torch.where(held, u, 0.0)
    bs, f, l, h0 = b[some], first[some], last[some], s["h0"][some]
    a_first = a[bs, f]
    u[bs, f] += a_first * h0
    a[bs, f] = 0.0
    h = _plain_scan(a, u)
    h_last = s["h0"].clone()
    h_last[some] = h[bs, l]
    out = h.reshape(s["x"].shape).to(dtype), h_last
    if not train:
        return out
    dh = (s["dh"][None] if case["form"] == "packed" else s["dh"]).float()
    if held is not None:
        dh = torch.where(held, dh, 0.0)
    dh = dh.clone()
    dh[bs, l] += s["dlast"][some]
    back = _plain_scan(a.flip(1), (a * dh).flip(1)).flip(1)  # a_t r_t, zero in front of each sequence
    r = dh.clone()
    r[:, :-1] += back[:, 1:]
    before = torch.zeros_like(h)
    before[:, 1:] = h[:, :-1]
    before[bs, f] = h0
    if case["drive"] == "complement":
        dx, da = r * rest, r * (before - x)
    else:
        dx, da = r, r * before
    dgate = da * slope
    if held is not None:
        dx, dgate = torch.where(held, dx, 0.0), torch.where(held, dgate, 0.0)
    dh0 = s["dlast"].clone()
    dh0[some] = a_first * r[bs, f]
    return out + (dx.reshape(s["x"].shape).to(dtype), dgate.reshape(s["x"].shape).to(dtype), dh0)


def _plain_step(case, s):
    a, _, u, _, _ = _plain_terms(case, s["x"], s["gate"])
    on = s["slots"] >= 0
    at = s["slots"].long().clamp(min=0)
    h = torch.where(on[:, None], a * s["state"][at] + u, 0.0)
    at = torch.where(on, at, s["state"].shape[0])  # idle places write to a row that is cut off
    wide = torch.cat([s["state"], s["state"][:1]])
    wide[at] = h
    s["state"].copy_(wide[:-1])
    return h.to(s["x"].dtype), s["state"]


def _plain_norm(case, s, train):
    dtype, shape = s["x"].dtype, s["x"].shape
    n, S, G, D = case["batch"], case["rows"], case["groups"], case["width"]
    x = s["x"].float().reshape(n, S, G, D)
    w, b = s["weight"].reshape(G, D), s["bias"].reshape(G, D)
    held, count = None, float(S * D)
    if s["lengths"] is not None:
        held = (torch.arange(S, device="cuda")[None, :] < s["lengths"][:, None])[:, :, None, None]
        count = (s["lengths"].float() * D).clamp(min=1.0)[:, None, None, None]
        x = torch.where(held, x, 0.0)
    mean = x.sum((1, 3), keepdim=True) / count
    off = x - mean
    if held is not None:
        off = torch.where(held, off, 0.0)
    rstd = torch.rsqrt((off * off).sum((1, 3), keepdim=True) / count + EPS)
    xhat = off * rstd
    z = xhat * w + b
    act = case["activation"]
    if act == "silu":
        p = torch.sigmoid(z)
        y = z * p
    elif act == "gelu":
        p = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        y = z * p
    else:
        y = z
    if held is not None:
        y = torch.where(held, y, 0.0)
    y = y.reshape(shape).to(dtype)
    if not train:
        return y
    dz = s["dy"].float().reshape(n, S, G, D)
    if act == "silu":
        dz = dz * (p * (1.0 + z * (1.0 - p)))
    elif act == "gelu":
        dz = dz * (p + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi)))
    if held is not None:
        dz = torch.where(held, dz, 0.0)
    db, dw = dz.sum((0, 1)).reshape(-1), (dz * xhat).sum((0, 1)).reshape(-1)
    t = dz * w
    m1 = t.sum((1, 3), keepdim=True) / count
    m2 = (t * xhat).sum((1, 3), keepdim=True) / count
    dx = rstd * (t - m1 - xhat * m2)
    if held is not None:
        dx = torch.where(held, dx, 0.0)
    return y, dx.reshape(shape).to(dtype), dw, db


def run(s):
    case = s["case"]
    op = case["op"]
    train = op.endswith("train")
    if not own:
        if op == "step":
            return _plain_step(case, s)
        return _plain_recurrence(case, s, train) if op.startswith("scan") else _plain_norm(case, s, train)
    import fft_block_toeplitz_amd as fm

    if op == "step":
        h = fm.recurrence_step(s["x"], s["gate"], s["state"], s["slots"], decay=case["decay"], drive=case["drive"])
        return h, s["state"]
    if op.startswith("scan"):
        how = {"decay": case["decay"], "drive": case["drive"], "lengths": s["lengths"], "offsets": s["offsets"]}
        if not train:
            return fm.recurrence(s["x"], s["gate"], s["h0"], **how)
        h, last, carries = fm.recurrence(s["x"], s["gate"], s["h0"], save=True, **how)
        return (h, last) + fm.recurrence_backward(s["dh"], s["x"], s["gate"], carries, s["h0"], s["dlast"], **how)
    how = {"activation": None if case["activation"] == "none" else case["activation"], "lengths": s["lengths"]}
    if not train:
        return fm.group_norm(s["x"], case["groups"], s["weight"], s["bias"], eps=EPS, **how)
    y, stats = fm.group_norm(s["x"], case["groups"], s["weight"], s["bias"], eps=EPS, save=True, **how)
    return (y,) + fm.group_norm_backward(s["dy"], s["x"], stats, case["groups"], s["weight"], s["bias"], **how)


# ------------------------------------------------------------ in 64 bits
def _exact_gate(case, g):
    """The decay in 64 bits and its slope."""
    if case["decay"] == "sigmoid":
        a = 1.0 / (1.0 + torch.exp(-g))
        return a, a * (1.0 - a)
    return (g.exp(), g.exp()) if case["decay"] == "exp" else (g, torch.ones_like(g))


def _exact_recurrence(case, s, train):
    """The definition step by step. Each sequence is a row of a padded batch; where a row has ended its state stays."""
    x, g = s["x"].double(), s["gate"].double()
    dh = s["dh"].double() if train else None
    n, C = case["batch"], case["channels"]
    spans = [(0, case["steps"])] * n
    if case["form"] == "padded":
        spans = [(0, int(v)) for v in s["lengths"].tolist()]
    elif case["form"] == "packed":
        o = s["offsets"].tolist()
        spans = list(zip(o[:-1], o[1:]))
    longest = max(e - b for b, e in spans)

    def rows(t):  # [longest, n, C]
        if case["form"] == "batch":
            return t.transpose(0, 1)
        p = torch.zeros((longest, n, C), dtype=torch.float64, device="cuda")
        for i, (b, e) in enumerate(spans):
            p[:e - b, i] = t[b:e] if case["form"] == "packed" else t[i, :e]
        return p

    def back(p):
        if case["form"] == "batch":
            return p.transpose(0, 1)
        t = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
        for i, (b, e) in enumerate(spans):
            if case["form"] == "packed":
                t[b:e] = p[:e - b, i]
            else:
                t[i, :e] = p[:e, i]
        return t

    on = torch.tensor([[float(k < e - b) for b, e in spans] for k in range(longest)], dtype=torch.float64)
    on = on.cuda().reshape(longest, n, 1)
    x, g = rows(x), rows(g)
    a, slope = _exact_gate(case, g)
    u = (1.0 - a) * x if case["drive"] == "complement" else x
    keep = 1.0 - on  # an ended row: h stays
    a_on, u_on = a * on + keep, u * on
    h = torch.empty((longest + 1, n, C), dtype=torch.float64, device="cuda")
    h[0] = s["h0"]
    for k in range(longest):
        torch.addcmul(u_on[k], a_on[k], h[k], out=h[k + 1])
    out = back(h[1:] * on), h[longest].clone()
    if not train:
        return out
    d = rows(dh) * on
    r = s["dlast"].double()  # the gradient of the state after step k
    dx, dg = torch.zeros_like(x), torch.zeros_like(x)
    for k in range(longest - 1, -1, -1):
        r = r + d[k]
        dx[k] = r
        r = r * a_on[k]
    real = dx * on
    if case["drive"] == "complement":
        dg = real * (h[:-1] - x) * slope
        dx = real * (1.0 - a)
    else:
        dg = real * h[:-1] * slope
        dx = real
    return out + (back(dx), back(dg), r)


def _exact_step(case, s):
    x, g, state = s["x"].double(), s["gate"].double(), s["state"].double()
    a, _ = _exact_gate(case, g)
    h = torch.zeros_like(x)
    for i, k in enumerate(s["slots"].tolist()):
        if k >= 0:
            state[k] = a[i] * state[k] + ((1.0 - a[i]) * x[i] if case["drive"] == "complement" else x[i])
            h[i] = state[k]
    return h, state


def _exact_norm(case, s, train):
    """Sample by sample from the definition, the gradients by automatic differentiation in 64 bits."""
    n, S, G, D = case["batch"], case["rows"], case["groups"], case["width"]
    x = s["x"].double().requires_grad_(train)
    w, b = s["weight"].double().requires_grad_(train), s["bias"].double().requires_grad_(train)

    def whole(v, m):  # v: [samples, rows, C] without padding
        v = v.reshape(v.shape[0], m, G, D)
        var, mean = torch.var_mean(v, (1, 3), correction=0, keepdim=True)
        z = ((v - mean) / torch.sqrt(var + EPS)).reshape(v.shape[0], m, G * D) * w + b
        if case["activation"] == "silu":
            return z / (1.0 + torch.exp(-z))
        if case["activation"] == "gelu":
            return 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
        return z

    if s["lengths"] is None:
        y = whole(x.reshape(n, S, G * D), S).reshape(x.shape)
    else:
        y = torch.zeros_like(x)
        for i, m in enumerate(s["lengths"].tolist()):
            if m > 0:
                y[i, :m] = whole(x[i:i + 1, :m], m)[0]
    if not train:
        return y.detach()
    if not y.requires_grad:  # no sample holds a row
        return y, torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(b)
    grads = torch.autograd.grad(y, (x, w, b), s["dy"].double())
    return (y.detach(),) + grads


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "step":
        return _exact_step(case, s)
    if op.startswith("scan"):
        return _exact_recurrence(case, s, op.endswith("train"))
    return _exact_norm(case, s, op.endswith("train"))
