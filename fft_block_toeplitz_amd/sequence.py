"""Sequence operators on torch tensors: a gated linear recurrence along time
(``recurrence``, ``recurrence_backward``, ``recurrence_step``) and group
normalisation with an activation over channels-last fields (``group_norm``,
``group_norm_backward``).

Like F, the recurrence is a causal linear operator along time on fields
[time][channels]; where F's blocks depend on i - j alone, its decays may
change at every step. With constant decays it is the block Toeplitz F with
F_k = diag(a^k).

Thin wrappers of the C entry points declared in ``include/fftmv.h``: they
check arguments, allocate outputs and pass pointers; torch supplies device
memory and streams. Elements are float32, bfloat16 or float16; states,
statistics and parameters are float32. ``layers`` holds the differentiable
forms. There is no fallback: without the built library every call raises.
"""

from __future__ import annotations

import ctypes
import functools

from . import FFTMV_SUCCESS, FftmvError, lib

FFTMV_F32, FFTMV_BF16, FFTMV_F16 = 0, 1, 2
FFTMV_RECURRENCE_CHUNK = 128
DECAYS = {"sigmoid": 0, "exp": 1, "value": 2}
DRIVES = {"complement": 0, "plain": 1}
ACTIVATIONS = {None: 0, "silu": 1, "gelu": 2}

_I64, _I32, _F32, _P, _Z = ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t


def _fields(text, kind):
    return [(name, kind) for name in text.split()]


class _Recurrence(ctypes.Structure):  # fftmv_recurrence_t
    _fields_ = (_fields("batch steps channels", _I64) + _fields("dtype decay drive", _I32)
                + [("call", ctypes.c_uint32)] + _fields("lengths offsets", _P)
                + [("x", _P), ("x_batch", _I64), ("x_step", _I64)]
                + [("gate", _P), ("gate_batch", _I64), ("gate_step", _I64)]
                + _fields("h0 carries", _P)
                + [("counters", _P), ("counter_bytes", _Z), ("workspace", _P), ("workspace_bytes", _Z)]
                + [("h", _P), ("h_batch", _I64), ("h_step", _I64), ("h_last", _P)]
                + [("dh", _P), ("dh_batch", _I64), ("dh_step", _I64), ("dh_last", _P)]
                + [("dx", _P), ("dx_batch", _I64), ("dx_step", _I64)]
                + [("dgate", _P), ("dgate_batch", _I64), ("dgate_step", _I64), ("dh0", _P)])


class _Step(ctypes.Structure):  # fftmv_recurrence_step_t
    _fields_ = (_fields("batch channels places", _I64) + _fields("dtype decay drive reserved", _I32)
                + [("x", _P), ("x_step", _I64), ("gate", _P), ("gate_step", _I64)]
                + [("state", _P), ("state_step", _I64), ("slots", _P), ("h", _P), ("h_step", _I64)])


class _GroupNorm(ctypes.Structure):  # fftmv_group_norm_t
    _fields_ = (_fields("samples rows channels groups", _I64) + _fields("dtype activation", _I32)
                + [("eps", _F32), ("reserved", _I32), ("lengths", _P)]
                + [("x", _P), ("x_sample", _I64), ("x_row", _I64)]
                + _fields("weight bias stats workspace", _P) + [("workspace_bytes", _Z)]
                + [("y", _P), ("y_sample", _I64), ("y_row", _I64)]
                + [("dy", _P), ("dy_sample", _I64), ("dy_row", _I64)]
                + [("dx", _P), ("dx_sample", _I64), ("dx_row", _I64)]
                + _fields("dweight dbias", _P))


# ---- same-name wrappers of the C entry points (structures, streams as ints)
_bound = None


def _lib():
    global _bound
    if _bound is None:
        L = lib()
        Z = ctypes.POINTER(_Z)
        L.fftmv_recurrence_sizes.argtypes = [_I64, _I64, _I64, ctypes.c_int, ctypes.POINTER(_I64), Z, Z]
        L.fftmv_group_norm_workspace.argtypes = [_I64, _I64, _I64, _I64, Z]
        for name, kind in (("recurrence_forward", _Recurrence), ("recurrence_backward", _Recurrence),
                           ("recurrence_step", _Step), ("group_norm_forward", _GroupNorm),
                           ("group_norm_backward", _GroupNorm)):
            getattr(L, "fftmv_" + name).argtypes = [ctypes.POINTER(kind), _P]
        _bound = L
    return _bound


def _check(status, what):
    if status != FFTMV_SUCCESS:
        raise FftmvError(status, what)


def fftmv_recurrence_sizes(batch: int, steps: int, channels: int, packed: bool) -> tuple[int, int, int]:
    """(rows of carries, bytes of counters, bytes of workspace) of a forward or backward call."""
    c, n, m = _I64(), _Z(), _Z()
    _check(_lib().fftmv_recurrence_sizes(batch, steps, channels, packed, ctypes.byref(c), ctypes.byref(n),
                                         ctypes.byref(m)), "fftmv_recurrence_sizes")
    return c.value, n.value, m.value


def fftmv_recurrence_forward(r: _Recurrence, stream: int = 0) -> None:
    _check(_lib().fftmv_recurrence_forward(r, stream), "fftmv_recurrence_forward")


def fftmv_recurrence_backward(r: _Recurrence, stream: int = 0) -> None:
    _check(_lib().fftmv_recurrence_backward(r, stream), "fftmv_recurrence_backward")


def fftmv_recurrence_step(r: _Step, stream: int = 0) -> None:
    _check(_lib().fftmv_recurrence_step(r, stream), "fftmv_recurrence_step")


def fftmv_group_norm_workspace(samples: int, rows: int, channels: int, groups: int) -> int:
    n = _Z()
    _check(_lib().fftmv_group_norm_workspace(samples, rows, channels, groups, ctypes.byref(n)),
           "fftmv_group_norm_workspace")
    return n.value


def fftmv_group_norm_forward(g: _GroupNorm, stream: int = 0) -> None:
    _check(_lib().fftmv_group_norm_forward(g, stream), "fftmv_group_norm_forward")


def fftmv_group_norm_backward(g: _GroupNorm, stream: int = 0) -> None:
    _check(_lib().fftmv_group_norm_backward(g, stream), "fftmv_group_norm_backward")


# ---- argument checks shared by the torch layer
_types = None


def _torch_types():
    global _types
    import torch

    _types = {torch.float32: FFTMV_F32, torch.bfloat16: FFTMV_BF16, torch.float16: FFTMV_F16}
    return _types


def _dtype_of(x, name):
    import torch

    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    code = (_types or _torch_types()).get(x.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, got {x.dtype}")
    if x.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} is on {x.device}, not on the current device")
    return code


def _field(t, like, name):
    """(pointer, batch stride, step stride) of a channels-last field of the shape, type and device of ``like``."""
    if t.shape != like.shape or t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{name} must have the shape, type and device of its counterpart: got {tuple(t.shape)} "
                         f"{t.dtype} on {t.device}, expected {tuple(like.shape)} {like.dtype} on {like.device}")
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] != 1 and t.numel():
        raise ValueError(f"{name}: channels must be contiguous (stride 1), got strides {st}")
    return (t.data_ptr(), st[0] if len(st) == 3 else 0, st[-2])


def _floats(t, shape, like, name):
    """Pointer of an optional contiguous float32 tensor."""
    if t is None:
        return None
    import torch

    if t.dtype != torch.float32 or tuple(t.shape) != shape or not t.is_contiguous() or t.device != like.device:
        raise ValueError(f"{name} must be a contiguous float32 tensor {shape} on {like.device}, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


def _ints(t, n, like, name):
    if t is None:
        return None
    import torch

    if t.dtype != torch.int32 or tuple(t.shape) != (n,) or not t.is_contiguous() or t.device != like.device:
        raise ValueError(f"{name} must be a contiguous int32 tensor ({n},) on {like.device}, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


def _choice(value, table, name):
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{name} must be one of {[k for k in table]}, got {value!r}") from None


def _span(t):
    """First byte and the byte after the last of a strided tensor."""
    n = sum((s - 1) * st for s, st in zip(t.shape, t.stride())) + 1 if t.numel() else 0
    return t.data_ptr(), t.data_ptr() + n * t.element_size()


def _output(out, like, inputs, name):
    """A new contiguous tensor like ``like``, or ``out`` after its checks."""
    import torch

    if out is None:
        return torch.empty(like.shape, dtype=like.dtype, device=like.device)
    if out.shape != like.shape or out.dtype != like.dtype or out.device != like.device or not out.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {like.dtype} tensor {tuple(like.shape)} on {like.device}")
    lo, hi = _span(out)
    for t in inputs:
        if t is not None:
            a, b = _span(t)
            if a < hi and lo < b:
                raise ValueError(f"{name} must not overlap an input")
    return out


class _On:
    """The stream that a call runs on: allocations inside belong to it, and
    tensors that came from another stream are kept for it."""

    def __init__(self, stream, *tensors):
        self.stream, self.tensors, self.inside = stream, tensors, None

    def __enter__(self):
        import torch

        if self.stream is None:
            return torch.cuda.current_stream().cuda_stream
        if self.stream != torch.cuda.current_stream():
            self.inside = torch.cuda.stream(self.stream)
            self.inside.__enter__()
            for t in self.tensors:
                if t is not None:
                    t.record_stream(self.stream)
        return self.stream.cuda_stream

    def __exit__(self, *what):
        if self.inside is not None:
            self.inside.__exit__(*what)


# ---- the recurrence
_workspaces = {}
_sizes = functools.lru_cache(maxsize=1024)(fftmv_recurrence_sizes)  # a function of the shape alone


def _workspace(sizes, stream, like):
    """(counters' address and bytes, workspace's address and bytes, number of
    the call on it). Calls of one stream share a workspace, which is kept and
    grown; a call under graph capture gets memory of the graph's own, cleared
    inside the graph."""
    import torch

    _, few, many = sizes
    if many == 0:
        return None, 0, None, 0, 0
    new = lambda n: torch.zeros(n, dtype=torch.uint8, device=like.device)  # noqa: E731
    if torch.cuda.is_current_stream_capturing():
        w = [new(few), new(many), 0]
    else:
        w = _workspaces.get((like.get_device(), stream))
        if w is None or w[0].numel() < few or w[1].numel() < many:
            if w is not None:
                few, many = max(few, w[0].numel()), max(many, w[1].numel())
            w = _workspaces[like.get_device(), stream] = [new(few), new(many), 0]
        elif w[2] == 2 ** 32 - 1:
            w[1].zero_()
            w[2] = 0
    w[2] += 1
    return w[0].data_ptr(), w[0].numel(), w[1].data_ptr(), w[1].numel(), w[2]


def _sequences(x, lengths, offsets):
    """(batch, steps, channels) of the three forms."""
    if offsets is not None:
        if lengths is not None:
            raise ValueError("lengths belong to padded batches and offsets to packed ones: give one of them")
        if x.dim() != 2 or offsets.dim() != 1 or offsets.shape[0] < 1:
            raise ValueError(f"a packed field is [steps, channels] with offsets [sequences + 1], got "
                             f"{tuple(x.shape)} and {tuple(offsets.shape)}")
        T, C = x.shape
        return offsets.shape[0] - 1, T, C
    if x.dim() == 3:
        B, T, C = x.shape
    elif x.dim() == 2:
        (T, C), B = x.shape, 1
    else:
        raise ValueError(f"x must be [batch, steps, channels] or [steps, channels], got {tuple(x.shape)}")
    return B, T, C


def recurrence(x, gate, h0=None, *, decay="sigmoid", drive="complement", lengths=None, offsets=None, save=False,
               out=None, stream=None):
    """Gated linear recurrence along time, per sequence and channel:

        h_t = a_t h_{t-1} + u_t,   h_{-1} = h0 (zeros when None)

    ``decay``: a = sigmoid(gate) ("sigmoid"), exp(gate) ("exp") or gate
    ("value"); ``drive``: u = (1 - a) x ("complement") or x ("plain").
    x and gate are [batch, steps, channels] (or one sequence [steps,
    channels]) with contiguous channels and any strides otherwise.
    ``lengths`` (int32 [batch]): padded batch, steps from lengths[b] on are
    not read and come back zero. ``offsets`` (int32 [sequences + 1]): x is
    [steps, channels], sequence b its rows offsets[b]..offsets[b+1]-1; rows
    of no sequence come back zero.

    Returns h (x's type) and the last states, float32 [batch, channels];
    with ``save`` also the carries that ``recurrence_backward`` needs. Runs
    on ``stream`` (default: the current one), without synchronising."""
    import torch

    dtype = _dtype_of(x, "x")
    B, T, C = _sequences(x, lengths, offsets)
    kinds = _choice(decay, DECAYS, "decay"), _choice(drive, DRIVES, "drive")
    xf, gf = _field(x, x, "x"), _field(gate, x, "gate")
    h0p = _floats(h0, (B, C), x, "h0")
    lens, offs = _ints(lengths, B, x, "lengths"), _ints(offsets, B + 1, x, "offsets")
    with _On(stream, x, gate, h0, lengths, offsets, out) as s:
        h = _output(out, x, (x, gate), "out")
        last = torch.empty((B, C), dtype=torch.float32, device=x.device)
        if B == 0:
            if T:
                h.zero_()
            return (h, last, torch.empty((0, C), device=x.device)) if save else (h, last)
        sizes = _sizes(B, T, C, offsets is not None)
        carries = torch.empty((sizes[0], C), dtype=torch.float32, device=x.device) if save else None
        *ws, call = _workspace(sizes, s, x)
        r = _Recurrence(B, T, C, dtype, *kinds, call, lens, offs, *xf, *gf, h0p, carries.data_ptr() if save else None,
                        *ws, *_field(h, x, "out"), last.data_ptr())
        fftmv_recurrence_forward(r, s)
    return (h, last, carries) if save else (h, last)


def recurrence_backward(dh, x, gate, carries, h0=None, dh_last=None, *, decay="sigmoid", drive="complement",
                        lengths=None, offsets=None, stream=None):
    """Gradients of ``recurrence``: (dx, dgate, dh0) from dh, the gradient of
    h, and dh_last, that of the last states (zeros when None). x, gate, h0
    and the keywords are the forward call's, ``carries`` what it saved; h is
    recomputed from them in float32."""
    import torch

    dtype = _dtype_of(x, "x")
    B, T, C = _sequences(x, lengths, offsets)
    kinds = _choice(decay, DECAYS, "decay"), _choice(drive, DRIVES, "drive")
    xf, gf, df = _field(x, x, "x"), _field(gate, x, "gate"), _field(dh, x, "dh")
    h0p, lp = _floats(h0, (B, C), x, "h0"), _floats(dh_last, (B, C), x, "dh_last")
    sizes = _sizes(B, T, C, offsets is not None) if B else (0, 0, 0)
    if carries is None:
        raise ValueError("carries must be what recurrence(..., save=True) returned")
    cp = _floats(carries, (sizes[0], C), x, "carries")
    lens, offs = _ints(lengths, B, x, "lengths"), _ints(offsets, B + 1, x, "offsets")
    with _On(stream, dh, x, gate, carries, h0, dh_last, lengths, offsets) as s:
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dg = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dh0 = torch.empty((B, C), dtype=torch.float32, device=x.device)
        if B == 0:
            if T:
                dx.zero_(), dg.zero_()
            return dx, dg, dh0
        *ws, call = _workspace(sizes, s, x)
        r = _Recurrence(B, T, C, dtype, *kinds, call, lens, offs, *xf, *gf, h0p, cp, *ws,
                        None, 0, 0, None, *df, lp, *_field(dx, x, "dx"), *_field(dg, x, "dgate"), dh0.data_ptr())
        fftmv_recurrence_backward(r, s)
    return dx, dg, dh0


def recurrence_step(x, gate, state, slots=None, *, decay="sigmoid", drive="complement", out=None, stream=None):
    """One time step of many streams against a cache of states, in place.
    x, gate: [batch, channels]; state: float32 [places, channels]; slots:
    int32 [batch], the place of each stream (None: stream b has place b). A
    slot outside the cache, -1 say, marks an idle stream: zeros come back
    and no state changes. Slots of one call must differ. Returns h [batch,
    channels]."""
    import torch

    dtype = _dtype_of(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x must be [batch, channels], got {tuple(x.shape)}")
    B, C = x.shape
    kinds = _choice(decay, DECAYS, "decay"), _choice(drive, DRIVES, "drive")
    xf, gf = _field(x, x, "x"), _field(gate, x, "gate")
    if state.dtype != torch.float32 or state.dim() != 2 or state.shape[1] != C or state.device != x.device or (
            state.stride(1) != 1 and C != 1) or (state.stride(0) < C and state.shape[0] > 1):
        raise ValueError(f"state must be a float32 tensor [places, {C}] on {x.device} with contiguous channels, got "
                         f"{tuple(state.shape)} {state.dtype}, strides {state.stride()}, on {state.device}")
    if slots is None and B > state.shape[0]:
        raise ValueError(f"{B} streams without slots need as many places, the state has {state.shape[0]}")
    sp = _ints(slots, B, x, "slots")
    with _On(stream, x, gate, state, slots, out) as s:
        h = _output(out, x, (x, gate, state), "out")
        if B == 0:
            return h
        if state.shape[0] == 0:
            return h.zero_()
        r = _Step(B, C, state.shape[0], dtype, *kinds, 0, xf[0], xf[2], gf[0], gf[2], state.data_ptr(),
                  max(state.stride(0), C), sp, h.data_ptr(), C)
        fftmv_recurrence_step(r, s)
    return h


# ---- group normalisation
def _samples(x):
    """x as [samples, rows, channels], without a copy."""
    if x.dim() == 3:
        return x
    if x.dim() == 2:
        return x.unsqueeze(1)
    if x.dim() < 2:
        raise ValueError(f"x must be [samples, ..., channels], got {tuple(x.shape)}")
    try:
        return x.view(x.shape[0], -1, x.shape[-1]) if x.numel() else x.reshape(x.shape[0], -1, x.shape[-1])
    except RuntimeError:
        raise ValueError(f"the rows of x {tuple(x.shape)} with strides {x.stride()} are not evenly spaced: "
                         "make it contiguous") from None


def group_norm(x, groups, weight=None, bias=None, *, eps=1e-5, activation=None, lengths=None, save=False, out=None,
               stream=None):
    """Group normalisation with an activation, channels last:

        y = act((x - mean) rstd weight + bias),   rstd = 1 / sqrt(var + eps)

    x: [samples, ..., channels] ([samples, channels]: every token by
    itself); mean and biased variance over all of a sample's rows and each
    of ``groups`` runs of neighbouring channels. weight, bias: float32
    [channels] or None. ``activation``: None, "silu" or "gelu" (exact).
    ``lengths`` (int32 [samples]): sample n holds its first lengths[n] rows;
    the others enter no sum, are not read, and come back zero.

    Returns y (x's type); with ``save`` also the statistics, float32
    [samples, groups, 2] (mean, rstd), that ``group_norm_backward`` needs."""
    import torch

    dtype = _dtype_of(x, "x")
    v = _samples(x)
    N, S, C = v.shape
    if not isinstance(groups, int) or groups < 1 or C < 1 or C % groups:
        raise ValueError(f"groups must divide the channels: got {groups!r} for {C}")
    act = _choice(activation, ACTIVATIONS, "activation")
    if not eps >= 0.0:
        raise ValueError(f"eps must be >= 0, got {eps}")
    xf = _field(v, v, "x")
    wp, bp = _floats(weight, (C,), x, "weight"), _floats(bias, (C,), x, "bias")
    lens = _ints(lengths, N, x, "lengths")
    with _On(stream, x, weight, bias, lengths, out) as s:
        y = _output(out, x, (x,), "out")
        stats = torch.empty((N, groups, 2), dtype=torch.float32, device=x.device) if save else None
        if N == 0:
            return (y, stats) if save else y
        need = fftmv_group_norm_workspace(N, S, C, groups)
        ws = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
        g = _GroupNorm(N, S, C, groups, dtype, act, eps, 0, lens, *xf, wp, bp, stats.data_ptr() if save else None,
                       ws.data_ptr() if need else None, need, y.data_ptr(), S * C, C)
        fftmv_group_norm_forward(g, s)
    return (y, stats) if save else y


def group_norm_backward(dy, x, stats, groups, weight=None, bias=None, *, activation=None, lengths=None, stream=None):
    """Gradients of ``group_norm``: (dx, dweight, dbias), the last two float32
    [channels], from dy, the gradient of y. x, the parameters and the
    keywords are the forward call's, ``stats`` what it saved."""
    import torch

    dtype = _dtype_of(x, "x")
    v = _samples(x)
    N, S, C = v.shape
    if not isinstance(groups, int) or groups < 1 or C < 1 or C % groups:
        raise ValueError(f"groups must divide the channels: got {groups!r} for {C}")
    act = _choice(activation, ACTIVATIONS, "activation")
    if dy.shape != x.shape:
        raise ValueError(f"dy must have x's shape {tuple(x.shape)}, got {tuple(dy.shape)}")
    xf, df = _field(v, v, "x"), _field(_samples(dy), v, "dy")
    wp, bp = _floats(weight, (C,), x, "weight"), _floats(bias, (C,), x, "bias")
    sp = _floats(stats, (N, groups, 2), x, "stats")
    if sp is None:
        raise ValueError("stats must be what group_norm(..., save=True) returned")
    lens = _ints(lengths, N, x, "lengths")
    with _On(stream, dy, x, stats, weight, bias, lengths) as s:
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        if N == 0:
            return dx, torch.zeros(C, device=x.device), torch.zeros(C, device=x.device)
        dw = torch.empty(C, dtype=torch.float32, device=x.device)
        db = torch.empty(C, dtype=torch.float32, device=x.device)
        need = fftmv_group_norm_workspace(N, S, C, groups)
        ws = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
        g = _GroupNorm(N, S, C, groups, dtype, act, 0.0, 0, lens, *xf, wp, bp, sp, ws.data_ptr() if need else None,
                       need, None, 0, 0, *df, dx.data_ptr(), S * C, C, dw.data_ptr(), db.data_ptr())
        fftmv_group_norm_backward(g, s)
    return dx, dw, db
