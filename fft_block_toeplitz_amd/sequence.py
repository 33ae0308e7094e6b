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
statistics and parameters are float32. ``recurrence`` and ``group_norm`` of
tensors that require a gradient go through the differentiable forms in
``layers``; with ``save=True`` they are the first half of a gradient taken by
hand, and their results carry none. There is no fallback: without the built
library every call raises.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import struct
import threading

from . import FFTMV_SUCCESS, FftmvError, lib

FFTMV_F32, FFTMV_BF16, FFTMV_F16 = 0, 1, 2
FFTMV_RECURRENCE_CHUNK = 128
DECAYS = {"sigmoid": 0, "exp": 1, "value": 2}
DRIVES = {"complement": 0, "plain": 1}
ACTIVATIONS = {None: 0, "silu": 1, "gelu": 2}

# The structures of include/fftmv.h as packed bytes, fields in their order (q:
# int64, i / I: int32, f: float, P: pointer, N: size_t; native alignment). A
# bytes object is a quarter of the cost of a ctypes structure, and these calls
# answer single time steps.
_RECURRENCE = struct.Struct("@3q3iI2P PqqPqq2P PNPN PqqP PqqP PqqPqqP")  # fftmv_recurrence_t
_STEP = struct.Struct("@3q4i PqPq PqP Pq")  # fftmv_recurrence_step_t
_GROUP_NORM = struct.Struct("@4q2ifiP Pqq 4PN Pqq PqqPqq2P")  # fftmv_group_norm_t
_I64, _P, _Z = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t


# ---- same-name wrappers of the C entry points (structures as bytes, streams as ints)
_bound = None


def _lib():
    global _bound
    if _bound is None:
        L = lib()
        Z = ctypes.POINTER(_Z)
        L.fftmv_recurrence_sizes.argtypes = [_I64, _I64, _I64, ctypes.c_int, ctypes.POINTER(_I64), Z, Z]
        L.fftmv_group_norm_workspace.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int, ctypes.c_int, Z]
        for name in ("recurrence_forward", "recurrence_backward", "recurrence_step", "group_norm_forward",
                     "group_norm_backward"):
            getattr(L, "fftmv_" + name).argtypes = [ctypes.c_char_p, _P]
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


def fftmv_recurrence_forward(r: bytes, stream: int = 0) -> None:
    status = (_bound or _lib()).fftmv_recurrence_forward(r, stream)
    if status:
        _check(status, "fftmv_recurrence_forward")


def fftmv_recurrence_backward(r: bytes, stream: int = 0) -> None:
    status = (_bound or _lib()).fftmv_recurrence_backward(r, stream)
    if status:
        _check(status, "fftmv_recurrence_backward")


def fftmv_recurrence_step(r: bytes, stream: int = 0) -> None:
    status = (_bound or _lib()).fftmv_recurrence_step(r, stream)
    if status:
        _check(status, "fftmv_recurrence_step")


def fftmv_group_norm_workspace(samples: int, rows: int, channels: int, groups: int, dtype: int,
                               backward: bool) -> int:
    n = _Z()
    _check(_lib().fftmv_group_norm_workspace(samples, rows, channels, groups, dtype, backward, ctypes.byref(n)),
           "fftmv_group_norm_workspace")
    return n.value


def fftmv_group_norm_forward(g: bytes, stream: int = 0) -> None:
    status = (_bound or _lib()).fftmv_group_norm_forward(g, stream)
    if status:
        _check(status, "fftmv_group_norm_forward")


def fftmv_group_norm_backward(g: bytes, stream: int = 0) -> None:
    status = (_bound or _lib()).fftmv_group_norm_backward(g, stream)
    if status:
        _check(status, "fftmv_group_norm_backward")


# ---- argument checks shared by the torch layer
_torch = None
_types = {}


def _torch_module():
    """torch, imported by the first call."""
    global _torch
    if _torch is None:
        import torch

        _types.update({torch.float32: FFTMV_F32, torch.bfloat16: FFTMV_BF16, torch.float16: FFTMV_F16})
        _torch = torch
    return _torch


def _dtype_of(x, name):
    torch = _torch or _torch_module()
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    code = _types.get(x.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, got {x.dtype}")
    if x.get_device() != torch._C._cuda_getDevice():  # torch.cuda.current_device() without its check: x is there
        raise ValueError(f"{name} is on {x.device}, not on the current device")
    return code


def _differs(t, shape, like, name):
    return ValueError(f"{name} must have the shape, type and device of its counterpart: got {tuple(t.shape)} "
                      f"{t.dtype} on {t.device}, expected {tuple(shape)} {like.dtype} on {like.device}")


def _field(t, shape, like, name):
    """(pointer, batch stride, step stride) of a channels-last field of this shape, of ``like``'s type and device."""
    if t is not like and (t.shape != shape or t.dtype is not like.dtype or t.get_device() != like.get_device()):
        raise _differs(t, shape, like, name)
    st = t.stride()
    if st[-1] != 1 and shape[-1] != 1 and t.numel():
        raise ValueError(f"{name}: channels must be contiguous (stride 1), got strides {st}")
    return (t.data_ptr(), st[0] if len(st) == 3 else 0, st[-2])


def _floats(t, shape, like, name):
    """Pointer of an optional contiguous float32 tensor."""
    if t is None:
        return 0
    if t.dtype != _torch.float32 or t.shape != shape or not t.is_contiguous() or t.get_device() != like.get_device():
        raise ValueError(f"{name} must be a contiguous float32 tensor {shape} on {like.device}, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


def _ints(t, n, like, name):
    if t is None:
        return 0
    if t.dtype != _torch.int32 or t.shape != (n,) or not t.is_contiguous() or t.get_device() != like.get_device():
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
    if t.is_contiguous():
        return t.data_ptr(), t.data_ptr() + t.nbytes
    n = sum((s - 1) * st for s, st in zip(t.shape, t.stride())) + 1 if t.numel() else 0
    return t.data_ptr(), t.data_ptr() + n * t.element_size()


def _output(out, like, inputs):
    """A new contiguous tensor like ``like``, or ``out`` after its checks."""
    if out is None:
        return _torch.empty_like(like, memory_format=_torch.contiguous_format)
    if out.shape != like.shape or out.dtype != like.dtype or out.device != like.device or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {like.dtype} tensor {tuple(like.shape)} on {like.device}")
    lo, hi = _span(out)
    for t in inputs:
        if t is not None:
            a, b = _span(t)
            if a < hi and lo < b:
                raise ValueError("out must not overlap an input")
    return out


def _wants_grad(*tensors):
    """Autograd is on and one of these requires a gradient."""
    for t in tensors:
        if t is not None and t.requires_grad:
            return _torch.is_grad_enabled()
    return False


def _no_out(out):
    if out is not None:
        raise ValueError("out= takes results without a gradient: call under torch.no_grad() or detach the inputs")


def _wrote(*tensors):
    """What a kernel has written in place, through its address, counts as written for autograd too: a graph that has
    saved it raises in its backward pass instead of going on with other values."""
    _torch._C._increment_version(tensors)  # torch.autograd.graph.increment_version without its type check


class _On:
    """A stream that is not the current one: allocations inside belong to it,
    and tensors that came from another stream are kept for it."""

    def __init__(self, stream, *tensors):
        self.inside, self.stream, self.tensors = _torch.cuda.stream(stream), stream, tensors

    def __enter__(self):
        self.inside.__enter__()
        for t in self.tensors:
            if t is not None:
                t.record_stream(self.stream)

    def __exit__(self, *what):
        self.inside.__exit__(*what)


def _elsewhere(stream, call, *args, **kwargs):
    """The call with another stream current."""
    _torch_module()
    tensors = [t for t in (*args, *kwargs.values()) if isinstance(t, _torch.Tensor) and t.is_cuda]
    with _On(stream, *tensors):
        return call(*args, **kwargs)


def _current_stream(device):
    """Handle of the device's current stream (torch.cuda.current_stream builds an object first: 3 us)."""
    return _torch._C._cuda_getCurrentRawStream(device)


# ---- the recurrence
_workspaces = {}
_sizes = functools.lru_cache(maxsize=1024)(fftmv_recurrence_sizes)  # functions of the shape alone
_norm_sizes = functools.lru_cache(maxsize=1024)(fftmv_group_norm_workspace)


class _workspace:
    """The memory of one call, to be entered around its launch: (counters'
    address and bytes, workspace's address and bytes, number of the call on
    it). Calls of one stream share a workspace, which is kept and grown; a call
    under graph capture gets memory of the graph's own, cleared inside the
    graph. Threads may share a stream: a workspace is held until the call has
    been launched on it, so that none is replaced in front of a launch and
    numbers ascend in the order of the launches."""

    __slots__ = ("sizes", "device", "stream", "like", "held")
    lock = threading.Lock()

    def __init__(self, sizes, device, stream, like):
        self.sizes, self.device, self.stream, self.like = sizes, device, stream, like
        self.held = None

    def __enter__(self):
        _, few, many = self.sizes
        new = lambda n: _torch.zeros(n, dtype=_torch.uint8, device=self.like.device)  # noqa: E731
        if _torch.cuda.is_current_stream_capturing():
            a, b = self.held = new(few), new(many)
            return a.data_ptr(), few, b.data_ptr(), many, 1
        self.lock.acquire()
        try:
            w = _workspaces.get((self.device, self.stream))
            if w is None or w[1] < few or w[3] < many:
                if w is not None:
                    few, many = max(few, w[1]), max(many, w[3])
                a, b = new(few), new(many)
                w = _workspaces[self.device, self.stream] = [a.data_ptr(), few, b.data_ptr(), many, 0, a, b]
            elif w[4] == 2 ** 32 - 1:
                w[6].zero_()
                w[4] = 0
            w[4] += 1
        except BaseException:
            self.lock.release()
            raise
        self.held = self.lock
        return w[:5]

    def __exit__(self, *what):
        if self.held is self.lock:
            self.lock.release()
        self.held = None


_NO_WORKSPACE = contextlib.nullcontext((0, 0, 0, 0, 0))  # of a call whose sizes ask for none


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
    ``lengths`` (int32 [batch]): padded batch, steps from lengths[b] on do
    not matter and come back zero. ``offsets`` (int32 [sequences + 1]): x is
    [steps, channels], sequence b its rows offsets[b]..offsets[b+1]-1; rows
    of no sequence come back zero. Both are clamped to 0..steps.

    Returns h (x's type) and the last states, float32 [batch, channels],
    differentiable where x, gate or h0 requires a gradient; with ``save``
    without, but also the carries that ``recurrence_backward`` needs.
    Runs on ``stream`` (default: the current one), without synchronising."""
    if stream is not None:
        return _elsewhere(stream, recurrence, x, gate, h0, decay=decay, drive=drive, lengths=lengths, offsets=offsets,
                          save=save, out=out)
    dtype = _dtype_of(x, "x")
    if not save and _wants_grad(x, gate, h0, out):
        from . import layers

        _no_out(out)
        return layers.recurrence(x, gate, h0, decay=decay, drive=drive, lengths=lengths, offsets=offsets)
    B, T, C = _sequences(x, lengths, offsets)
    kinds = _choice(decay, DECAYS, "decay"), _choice(drive, DRIVES, "drive")
    shape, packed = x.shape, offsets is not None
    xf, gf = _field(x, shape, x, "x"), _field(gate, shape, x, "gate")
    h0p = _floats(h0, (B, C), x, "h0")
    lens, offs = _ints(lengths, B, x, "lengths"), _ints(offsets, B + 1, x, "offsets")
    h = _output(out, x, (x, gate, h0, lengths, offsets))
    last = x.new_empty((B, C), dtype=_torch.float32)
    if B == 0:
        h.zero_()
        return (h, last, last) if save else (h, last)
    sizes = _sizes(B, T, C, packed)
    carries = x.new_empty((sizes[0], C), dtype=_torch.float32) if save else None
    device = x.get_device()
    stream = _current_stream(device)
    with _workspace(sizes, device, stream, x) if sizes[2] else _NO_WORKSPACE as (*ws, call):
        r = _RECURRENCE.pack(B, T, C, dtype, *kinds, call, lens, offs, *xf, *gf, h0p,
                             carries.data_ptr() if save else 0, *ws, h.data_ptr(), T * C, C, last.data_ptr(), 0, 0, 0,
                             0, 0, 0, 0, 0, 0, 0, 0)
        fftmv_recurrence_forward(r, stream)
    if out is not None:
        _wrote(out)
    return (h, last, carries) if save else (h, last)


def recurrence_backward(dh, x, gate, carries, h0=None, dh_last=None, *, decay="sigmoid", drive="complement",
                        lengths=None, offsets=None, stream=None):
    """Gradients of ``recurrence``: (dx, dgate, dh0) from dh, the gradient of
    h, and dh_last, that of the last states (zeros when None). x, gate, h0
    and the keywords are the forward call's, ``carries`` what it saved; h is
    recomputed from them in float32."""
    if stream is not None:
        return _elsewhere(stream, recurrence_backward, dh, x, gate, carries, h0, dh_last, decay=decay, drive=drive,
                          lengths=lengths, offsets=offsets)
    dtype = _dtype_of(x, "x")
    B, T, C = _sequences(x, lengths, offsets)
    kinds = _choice(decay, DECAYS, "decay"), _choice(drive, DRIVES, "drive")
    shape = x.shape
    xf, gf, df = _field(x, shape, x, "x"), _field(gate, shape, x, "gate"), _field(dh, shape, x, "dh")
    h0p, lp = _floats(h0, (B, C), x, "h0"), _floats(dh_last, (B, C), x, "dh_last")
    sizes = _sizes(B, T, C, offsets is not None) if B else (0, 0, 0)
    if carries is None:
        raise ValueError("carries must be what recurrence(..., save=True) returned")
    cp = _floats(carries, (sizes[0], C), x, "carries")
    lens, offs = _ints(lengths, B, x, "lengths"), _ints(offsets, B + 1, x, "offsets")
    dx = _torch.empty_like(x, memory_format=_torch.contiguous_format)
    dg = _torch.empty_like(dx)
    dh0 = x.new_empty((B, C), dtype=_torch.float32)
    if B == 0:
        return dx.zero_(), dg.zero_(), dh0
    device = x.get_device()
    stream = _current_stream(device)
    with _workspace(sizes, device, stream, x) if sizes[2] else _NO_WORKSPACE as (*ws, call):
        r = _RECURRENCE.pack(B, T, C, dtype, *kinds, call, lens, offs, *xf, *gf, h0p, cp, *ws, 0, 0, 0, 0, *df, lp,
                             dx.data_ptr(), T * C, C, dg.data_ptr(), T * C, C, dh0.data_ptr())
        fftmv_recurrence_backward(r, stream)
    return dx, dg, dh0


def recurrence_step(x, gate, state, slots=None, *, decay="sigmoid", drive="complement", out=None,
                    stream=None):
    """One time step of many streams against a cache of states, in place.
    x, gate: [batch, channels]; state: float32 [places, channels]; slots:
    int32 [batch], the place of each stream (None: stream b has place b). A
    slot outside the cache, -1 say, marks an idle stream: zeros come back
    and no state changes. Slots of one call must differ. Returns h [batch,
    channels], which has no gradient: inputs that require one are refused
    unless autograd is off."""
    if stream is not None:
        return _elsewhere(stream, recurrence_step, x, gate, state, slots, decay=decay, drive=drive, out=out)
    dtype = _dtype_of(x, "x")
    if _wants_grad(x, gate, state, out):
        raise ValueError("a step in place has no gradient: call it under torch.no_grad(), or recurrence on whole series")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"x must be [batch, channels], got {tuple(shape)}")
    B, C = shape
    kinds = _choice(decay, DECAYS, "decay"), _choice(drive, DRIVES, "drive")
    xp, _, xs = _field(x, shape, x, "x")
    gp, _, gs = _field(gate, shape, x, "gate")
    places = state.shape[0] if state.dim() == 2 else -1
    ss = state.stride()
    if (places < 0 or state.dtype != _torch.float32 or state.shape[1] != C or state.get_device() != x.get_device()
            or (ss[1] != 1 and C != 1) or (ss[0] < C and places > 1)):
        raise ValueError(f"state must be a float32 tensor [places, {C}] on {x.device} with contiguous channels, got "
                         f"{tuple(state.shape)} {state.dtype}, strides {ss}, on {state.device}")
    if slots is None and B > places:
        raise ValueError(f"{B} streams without slots need as many places, the state has {places}")
    sp = _ints(slots, B, x, "slots")
    h = _output(out, x, (x, gate, state, slots))
    if B == 0 or places == 0:
        return h.zero_()
    fftmv_recurrence_step(_STEP.pack(B, C, places, dtype, *kinds, 0, xp, xs, gp, gs, state.data_ptr(),
                                     max(ss[0], C), sp, h.data_ptr(), C), _current_stream(x.get_device()))
    if out is None:
        _wrote(state)
    else:
        _wrote(state, out)
    return h


# ---- group normalisation
def _scratch(samples, rows, channels, groups, backward, like):
    """(scratch memory or None, its bytes) of a call of this shape."""
    need = _norm_sizes(samples, rows, channels, groups, _types[like.dtype], backward)
    return (like.new_empty(need, dtype=_torch.uint8), need) if need else (None, 0)


def _samples(x):
    """x as [samples, rows, channels], without a copy."""
    if x.dim() == 3:
        return x
    if x.dim() == 2:
        return x.unsqueeze(1)
    if x.dim() < 2:
        raise ValueError(f"x must be [samples, ..., channels], got {tuple(x.shape)}")
    try:
        return x.view(x.shape[0], math.prod(x.shape[1:-1]), x.shape[-1])
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
    the others enter no sum whatever they hold, and come back zero.

    Returns y (x's type), differentiable where x, weight or bias requires a
    gradient; with ``save`` without, but also the statistics, float32
    [samples, groups, 2] (mean, rstd), that ``group_norm_backward`` needs."""
    if stream is not None:
        return _elsewhere(stream, group_norm, x, groups, weight, bias, eps=eps, activation=activation, lengths=lengths,
                          save=save, out=out)
    dtype = _dtype_of(x, "x")
    if not save and _wants_grad(x, weight, bias, out):
        from . import layers

        _no_out(out)
        return layers.group_norm(x, groups, weight, bias, eps=eps, activation=activation, lengths=lengths)
    v = _samples(x)
    N, S, C = shape = v.shape
    if not isinstance(groups, int) or groups < 1 or C < 1 or C % groups:
        raise ValueError(f"groups must divide the channels: got {groups!r} for {C}")
    act = _choice(activation, ACTIVATIONS, "activation")
    if not eps >= 0.0:
        raise ValueError(f"eps must be >= 0, got {eps}")
    xf = _field(v, shape, v, "x")
    wp, bp = _floats(weight, (C,), x, "weight"), _floats(bias, (C,), x, "bias")
    lens = _ints(lengths, N, x, "lengths")
    y = _output(out, x, (x, weight, bias, lengths))
    stats = x.new_empty((N, groups, 2), dtype=_torch.float32) if save else None
    if N == 0:
        return (y, stats) if save else y
    ws, need = _scratch(N, S, C, groups, False, x)
    g = _GROUP_NORM.pack(N, S, C, groups, dtype, act, eps, 0, lens, *xf, wp, bp, stats.data_ptr() if save else 0,
                         ws.data_ptr() if need else 0, need, y.data_ptr(), S * C, C, 0, 0, 0, 0, 0, 0, 0, 0)
    fftmv_group_norm_forward(g, _current_stream(x.get_device()))
    if out is not None:
        _wrote(out)
    return (y, stats) if save else y


def group_norm_backward(dy, x, stats, groups, weight=None, bias=None, *, activation=None, lengths=None, stream=None):
    """Gradients of ``group_norm``: (dx, dweight, dbias), the last two float32
    [channels], from dy, the gradient of y. x, the parameters and the
    keywords are the forward call's, ``stats`` what it saved."""
    if stream is not None:
        return _elsewhere(stream, group_norm_backward, dy, x, stats, groups, weight, bias, activation=activation,
                          lengths=lengths)
    dtype = _dtype_of(x, "x")
    v = _samples(x)
    N, S, C = shape = v.shape
    if not isinstance(groups, int) or groups < 1 or C < 1 or C % groups:
        raise ValueError(f"groups must divide the channels: got {groups!r} for {C}")
    act = _choice(activation, ACTIVATIONS, "activation")
    if dy.shape != x.shape:
        raise ValueError(f"dy must have x's shape {tuple(x.shape)}, got {tuple(dy.shape)}")
    xf, df = _field(v, shape, v, "x"), _field(_samples(dy), shape, v, "dy")
    wp, bp = _floats(weight, (C,), x, "weight"), _floats(bias, (C,), x, "bias")
    if stats is None:
        raise ValueError("stats must be what group_norm(..., save=True) returned")
    sp = _floats(stats, (N, groups, 2), x, "stats")
    lens = _ints(lengths, N, x, "lengths")
    dx = _torch.empty_like(x, memory_format=_torch.contiguous_format)
    both = x.new_empty((2, C), dtype=_torch.float32)
    dw, db = both[0], both[1]
    if N == 0:
        both.zero_()
        return dx, dw, db
    ws, need = _scratch(N, S, C, groups, True, x)
    g = _GROUP_NORM.pack(N, S, C, groups, dtype, act, 0.0, 0, lens, *xf, wp, bp, sp, ws.data_ptr() if need else 0, need,
                         0, 0, 0, *df, dx.data_ptr(), S * C, C, dw.data_ptr(), db.data_ptr())
    fftmv_group_norm_backward(g, _current_stream(x.get_device()))
    return dx, dw, db
