"""The gated delta rule on torch tensors (``delta_rule``,
``delta_rule_backward``, ``delta_rule_step``) and the norms of its queries and
keys with a rotation by position (``qk_norm``, ``qk_norm_backward``).

The delta rule is a causal linear operator along time like ``recurrence``, with
a matrix for a state: per head it holds values under keys, answers queries from
them, and corrects what it holds under a key instead of adding to it. Queries
and keys are meant to be normalised (``qk_norm(..., norm="l2")``).

Thin wrappers of the C entry points declared in ``include/fftmv.h``, in the
manner of ``sequence``: elements are float32, bfloat16 or float16, one type for
all fields of a call; states and weights are float32. ``delta_rule`` and
``qk_norm`` of tensors that require a gradient go through the differentiable
forms in ``layers``. There is no fallback: without the built library every call
raises.
"""

from __future__ import annotations

import ctypes
import functools
import struct

from . import lib
from . import sequence as _sq
from .sequence import _check, _choice, _current_stream, _dtype_of, _elsewhere, _floats, _ints, _no_out, _no_tangents, \
    _output, _wants_grad, _wrote

FFTMV_DELTA_RUN = 64
FFTMV_DELTA_KEYS, FFTMV_DELTA_VALUES, FFTMV_QK_NORM_DIM = 128, 1024, 512
DECAYS = {"sigmoid": 0, "exp": 1}
RATES = {"sigmoid": 0, "value": 1}
NORMS = {"rms": 0, "l2": 1}
PAIRS = {"halves": 0, "neighbours": 1}

# the structures of include/fftmv.h as packed bytes; Pqqq: fftmv_heads_t
_DELTA = struct.Struct("@6q3if2P" + "Pqqq" * 5 + "3PN" + "PqqqP" * 2 + "Pqqq" * 5 + "P")  # fftmv_delta_rule_t
_DELTA_STEP = struct.Struct("@6q3if" + "Pqqq" * 5 + "PqP" + "Pqqq")  # fftmv_delta_rule_step_t
_QK_NORM = struct.Struct("@6q3if3Pq" + "Pqqq" * 2 + "2P" + "Pqqq" * 6 + "3PN")  # fftmv_qk_norm_t
_NONE = (0, 0, 0, 0)
_I64, _P, _Z = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
_bound = None


def _lib():
    global _bound
    if _bound is None:
        L = lib()
        L.fftmv_delta_rule_sizes.argtypes = [_I64] * 6 + [ctypes.c_int] * 3 + [ctypes.POINTER(_I64), ctypes.POINTER(_Z)]
        L.fftmv_qk_norm_workspace.argtypes = [_I64] * 5 + [ctypes.POINTER(_Z)]
        for name in ("delta_rule_forward", "delta_rule_backward", "delta_rule_step", "qk_norm_forward", "qk_norm_backward"):
            getattr(L, "fftmv_" + name).argtypes = [ctypes.c_char_p, _P]
        _bound = L
    return _bound


# ---- same-name wrappers of the C entry points (structures as bytes, streams as ints)
def fftmv_delta_rule_sizes(batch: int, steps: int, key_heads: int, heads: int, keys: int, values: int, dtype: int,
                           packed: bool, backward: bool) -> tuple[int, int]:
    """(runs of carries, bytes of workspace) of a forward or backward call."""
    n, m = _I64(), _Z()
    _check(_lib().fftmv_delta_rule_sizes(batch, steps, key_heads, heads, keys, values, dtype, packed, backward,
                                         ctypes.byref(n), ctypes.byref(m)), "fftmv_delta_rule_sizes")
    return n.value, m.value


def fftmv_delta_rule_forward(r: bytes, stream: int = 0) -> None:
    _check((_bound or _lib()).fftmv_delta_rule_forward(r, stream), "fftmv_delta_rule_forward")


def fftmv_delta_rule_backward(r: bytes, stream: int = 0) -> None:
    _check((_bound or _lib()).fftmv_delta_rule_backward(r, stream), "fftmv_delta_rule_backward")


def fftmv_delta_rule_step(r: bytes, stream: int = 0) -> None:
    _check((_bound or _lib()).fftmv_delta_rule_step(r, stream), "fftmv_delta_rule_step")


def fftmv_qk_norm_workspace(batch: int, steps: int, query_heads: int, key_heads: int, dim: int) -> int:
    n = _Z()
    _check(_lib().fftmv_qk_norm_workspace(batch, steps, query_heads, key_heads, dim, ctypes.byref(n)),
           "fftmv_qk_norm_workspace")
    return n.value


def fftmv_qk_norm_forward(n: bytes, stream: int = 0) -> None:
    _check((_bound or _lib()).fftmv_qk_norm_forward(n, stream), "fftmv_qk_norm_forward")


def fftmv_qk_norm_backward(n: bytes, stream: int = 0) -> None:
    _check((_bound or _lib()).fftmv_qk_norm_backward(n, stream), "fftmv_qk_norm_backward")


_sizes = functools.lru_cache(maxsize=1024)(fftmv_delta_rule_sizes)  # functions of the shape alone
_norm_bytes = functools.lru_cache(maxsize=1024)(fftmv_qk_norm_workspace)


# ---- argument checks
def _heads(t, shape, like, name):
    """(pointer, batch, step and head stride) of a field [batch, steps, heads, elements] or [steps, heads, elements] of
    ``like``'s type and device; gates are fields without the last axis."""
    if t is not like and (t.shape != shape or t.dtype is not like.dtype or t.get_device() != like.get_device()):
        raise _sq._differs(t, shape, like, name)
    st = t.stride()
    return (t.data_ptr(), *((0, *st) if len(st) == 2 else st[:3]))


def _elements(t, shape, like, name):
    """The same of fields with elements, which have to be contiguous."""
    if t is not like and (t.shape != shape or t.dtype is not like.dtype or t.get_device() != like.get_device()):
        raise _sq._differs(t, shape, like, name)
    st = t.stride()
    if st[-1] != 1 and shape[-1] != 1 and t.numel():
        raise ValueError(f"{name}: a head's elements must be contiguous (stride 1), got strides {st}")
    return (t.data_ptr(), *((0, *st[:2]) if len(st) == 3 else st[:3]))


def _shapes(q, k, v, gate, beta, offsets, lengths, step=False):
    """(batch, steps, key heads, heads, keys, values) after the checks that the five inputs fit together."""
    dims = 3 if step or offsets is not None else q.dim()
    if q.dim() != dims or dims not in (3, 4) or v.dim() != dims:
        raise ValueError("q, k and v are [batch, steps, heads, elements], or [steps, heads, elements] for one sequence or "
                         f"with offsets ([batch, heads, elements] for a step); got {tuple(q.shape)} and {tuple(v.shape)}")
    Hk, K = q.shape[-2:]
    H, V = v.shape[-2:]
    if q.shape[:-2] != v.shape[:-2]:
        raise ValueError(f"q and v must have the same rows: got {tuple(q.shape)} and {tuple(v.shape)}")
    if Hk < 1 or H % Hk or H < 1:
        raise ValueError(f"the heads of v must be a multiple of those of q and k: got {H} for {Hk}")
    if offsets is not None:
        if lengths is not None:
            raise ValueError("lengths belong to padded batches and offsets to packed ones: give one of them")
        if offsets.dim() != 1 or offsets.shape[0] < 1:
            raise ValueError(f"offsets must be [sequences + 1], got {tuple(offsets.shape)}")
        return offsets.shape[0] - 1, q.shape[0], Hk, H, K, V
    if step:
        return q.shape[0], 1, Hk, H, K, V
    return (q.shape[0] if dims == 4 else 1), q.shape[-3], Hk, H, K, V


def _inputs(q, k, v, gate, beta):
    """The five fields. (One after the other through the checks above takes twice the time, 3 us a call.)"""
    rows, dtype, device = v.shape[:-1], v.dtype, v.get_device()
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    if (k.shape != q.shape or gate.shape != rows or beta.shape != rows or q.dtype is not dtype or k.dtype is not dtype
            or gate.dtype is not dtype or beta.dtype is not dtype or q.get_device() != device or k.get_device() != device
            or gate.get_device() != device or beta.get_device() != device or qs[-1] != 1 or ks[-1] != 1 or vs[-1] != 1):
        return (*_elements(q, q.shape, v, "q"), *_elements(k, q.shape, v, "k"), *_elements(v, v.shape, v, "v"),
                *_heads(gate, rows, v, "gate"), *_heads(beta, rows, v, "beta"))
    if len(rows) == 3:
        return (q.data_ptr(), *qs[:3], k.data_ptr(), *ks[:3], v.data_ptr(), *vs[:3], gate.data_ptr(), *gate.stride(),
                beta.data_ptr(), *beta.stride())
    return (q.data_ptr(), 0, *qs[:2], k.data_ptr(), 0, *ks[:2], v.data_ptr(), 0, *vs[:2], gate.data_ptr(), 0,
            *gate.stride(), beta.data_ptr(), 0, *beta.stride())


def _empty(like):
    """A new contiguous tensor (new_empty(like.shape) takes half as long again)."""
    return _sq._torch.empty_like(like, memory_format=_sq._torch.contiguous_format)


def _fresh(t):
    """The field of a contiguous tensor with elements, or of a gate."""
    return t.data_ptr(), *((0, *t.stride()[:2]) if t.dim() == 3 else t.stride()[:3])


def _fresh_gate(t):
    return t.data_ptr(), *((0, *t.stride()) if t.dim() == 2 else t.stride())


def _scale(scale, keys):
    return keys ** -0.5 if scale is None else float(scale)


# ---- the delta rule
def delta_rule(q, k, v, gate, beta, h0=None, *, decay="sigmoid", rate="sigmoid", scale=None, lengths=None, offsets=None,
               save=False, out=None, stream=None):
    """Gated delta rule along time, per sequence and head, from S_{-1} = h0
    (zeros when None), a matrix [keys, values]:

        S_t = a_t S_{t-1} + b_t k_t (v_t - a_t S_{t-1}^T k_t)^T
        y_t = scale S_t^T q_t

    ``decay``: a = sigmoid(gate) ("sigmoid") or exp(gate) ("exp"; minus
    infinity clears the state, and decays are meant to be at most one: results
    are not finite where the gates of 64 steps add up to more than 88); ``rate``: b = sigmoid(beta) ("sigmoid") or
    beta ("value"); ``scale``: keys ** -0.5 when None. q, k: [batch, steps,
    key heads, keys] (or one sequence [steps, key heads, keys]), v: [batch,
    steps, heads, values], gate, beta: [batch, steps, heads], with contiguous
    elements and any strides otherwise. Heads are a multiple of key heads;
    neighbouring ones share queries and keys. keys <= 128, values <= 1024.
    ``lengths`` and ``offsets`` are those of ``recurrence``, rows of no
    sequence come back zero.

    Returns y (v's shape) and the last states, float32 [batch, heads, keys,
    values], differentiable where an input requires a gradient; with ``save``
    without, but also the carries that ``delta_rule_backward`` needs.
    Runs on ``stream`` (default: the current one), without synchronising."""
    if stream is not None:
        return _elsewhere(stream, delta_rule, q, k, v, gate, beta, h0, decay=decay, rate=rate, scale=scale,
                          lengths=lengths, offsets=offsets, save=save, out=out)
    dtype = _dtype_of(v, "v")
    _no_tangents(q, k, v, gate, beta, h0, out)
    if not save and _wants_grad(q, k, v, gate, beta, h0, out):
        from . import layers

        _no_out(out)
        return layers.delta_rule(q, k, v, gate, beta, h0, decay=decay, rate=rate, scale=scale, lengths=lengths,
                                 offsets=offsets)
    B, T, Hk, H, K, V = _shapes(q, k, v, gate, beta, offsets, lengths)
    kinds = _choice(decay, DECAYS, "decay"), _choice(rate, RATES, "rate")
    fields = _inputs(q, k, v, gate, beta)
    h0p = _floats(h0, (B, H, K, V), v, "h0")
    lens, offs = _ints(lengths, B, v, "lengths"), _ints(offsets, B + 1, v, "offsets")
    y = _output(out, v, (q, k, v, gate, beta, h0, lengths, offsets))
    last = v.new_empty((B, H, K, V), dtype=_sq._torch.float32)
    if B == 0:
        y.zero_()
        return (y, last, last.new_empty((0, H, K + FFTMV_DELTA_RUN, V))) if save else (y, last)
    runs, need = _sizes(B, T, Hk, H, K, V, dtype, offsets is not None, False)
    carries = v.new_empty((runs, H, K + FFTMV_DELTA_RUN, V), dtype=_sq._torch.float32) if save else None
    ws = v.new_empty(need, dtype=_sq._torch.uint8)
    r = _DELTA.pack(B, T, Hk, H, K, V, dtype, *kinds, _scale(scale, K), lens, offs, *fields, h0p,
                    carries.data_ptr() if save else 0, ws.data_ptr(), need, *_fresh(y), last.data_ptr(), *_NONE, 0,
                    *_NONE * 5, 0)
    fftmv_delta_rule_forward(r, _current_stream(v.get_device()))
    if out is not None:
        _wrote(out)
    return (y, last, carries) if save else (y, last)


def delta_rule_backward(dy, q, k, v, gate, beta, carries, h0=None, dh_last=None, *, decay="sigmoid", rate="sigmoid",
                        scale=None, lengths=None, offsets=None, stream=None):
    """Gradients of ``delta_rule``: (dq, dk, dv, dgate, dbeta, dh0) from dy, the
    gradient of y, and dh_last, that of the last states (zeros when None). The
    inputs and the keywords are the forward call's, ``carries`` what it saved."""
    if stream is not None:
        return _elsewhere(stream, delta_rule_backward, dy, q, k, v, gate, beta, carries, h0, dh_last, decay=decay,
                          rate=rate, scale=scale, lengths=lengths, offsets=offsets)
    dtype = _dtype_of(v, "v")
    _no_tangents(dy, q, k, v, gate, beta, carries, h0, dh_last)
    torch = _sq._torch
    B, T, Hk, H, K, V = _shapes(q, k, v, gate, beta, offsets, lengths)
    kinds = _choice(decay, DECAYS, "decay"), _choice(rate, RATES, "rate")
    fields, dyf = _inputs(q, k, v, gate, beta), _elements(dy, v.shape, v, "dy")
    h0p, lp = _floats(h0, (B, H, K, V), v, "h0"), _floats(dh_last, (B, H, K, V), v, "dh_last")
    runs, need = _sizes(B, T, Hk, H, K, V, dtype, offsets is not None, True) if B else (0, 0)
    if carries is None:
        raise ValueError("carries must be what delta_rule(..., save=True) returned")
    cp = _floats(carries, (runs, H, K + FFTMV_DELTA_RUN, V), v, "carries")
    lens, offs = _ints(lengths, B, v, "lengths"), _ints(offsets, B + 1, v, "offsets")
    dq, dk, dv, dg, db = (_empty(t) for t in (q, k, v, gate, beta))
    dh0 = v.new_empty((B, H, K, V), dtype=torch.float32)
    if B == 0:
        return dq.zero_(), dk.zero_(), dv.zero_(), dg.zero_(), db.zero_(), dh0
    ws = v.new_empty(need, dtype=torch.uint8)
    r = _DELTA.pack(B, T, Hk, H, K, V, dtype, *kinds, _scale(scale, K), lens, offs, *fields, h0p, cp, ws.data_ptr(),
                    need, *_NONE, 0, *dyf, lp, *_fresh(dq), *_fresh(dk), *_fresh(dv), *_fresh_gate(dg),
                    *_fresh_gate(db), dh0.data_ptr())
    fftmv_delta_rule_backward(r, _current_stream(v.get_device()))
    return dq, dk, dv, dg, db, dh0


def delta_rule_step(q, k, v, gate, beta, state, slots=None, *, decay="sigmoid", rate="sigmoid", scale=None, out=None,
                    stream=None):
    """One time step of many streams against a cache of states, in place. q, k:
    [batch, key heads, keys], v: [batch, heads, values], gate, beta: [batch,
    heads]; state: float32 [places, heads, keys, values], places any distance
    apart; slots: int32 [batch], as in ``recurrence_step`` (one outside the
    cache marks an idle stream: zeros come back and no state changes; slots of
    one call must differ). Returns y [batch, heads, values], which has no
    gradient: inputs that require one are refused unless autograd is off."""
    if stream is not None:
        return _elsewhere(stream, delta_rule_step, q, k, v, gate, beta, state, slots, decay=decay, rate=rate,
                          scale=scale, out=out)
    dtype = _dtype_of(v, "v")
    _no_tangents(q, k, v, gate, beta, state, out)
    if _wants_grad(q, k, v, gate, beta, state, out):
        raise ValueError("a step in place has no gradient: call it under torch.no_grad(), or delta_rule on whole series")
    B, _, Hk, H, K, V = _shapes(q, k, v, gate, beta, None, None, step=True)
    kinds = _choice(decay, DECAYS, "decay"), _choice(rate, RATES, "rate")
    # a row is a stream: batch strides are not used
    fields = _inputs(q, k, v, gate, beta)
    places = state.shape[0] if state.dim() == 4 else -1
    ss = state.stride()
    inner = H * K * V
    if (places < 0 or state.dtype != _sq._torch.float32 or state.shape[1:] != (H, K, V)
            or state.get_device() != v.get_device()
            or (ss[1:] != (K * V, V, 1) and places and not state[0].is_contiguous())
            or (ss[0] < inner and places > 1)):
        raise ValueError(f"state must be a float32 tensor [places, {H}, {K}, {V}] on {v.device}, each place contiguous, "
                         f"got {tuple(state.shape)} {state.dtype}, strides {ss}, on {state.device}")
    if slots is None and B > places:
        raise ValueError(f"{B} streams without slots need as many places, the state has {places}")
    sp = _ints(slots, B, v, "slots")
    y = _output(out, v, (q, k, v, gate, beta, state, slots))
    if B == 0 or places == 0:
        return y.zero_()
    r = _DELTA_STEP.pack(B, Hk, H, K, V, places, dtype, *kinds, _scale(scale, K), *fields, state.data_ptr(),
                         max(ss[0], inner), sp, *_fresh(y))
    fftmv_delta_rule_step(r, _current_stream(v.get_device()))
    if out is None:
        _wrote(state)
    else:
        _wrote(state, out)
    return y


# ---- norms of queries and keys
def _norm_call(q, k, q_weight, k_weight, norm, eps, frequencies, positions, pairs, lengths):
    """The head of the structure, up to the weights, and the sizes."""
    torch, shape, device = _sq._torch, tuple(q.shape), q.get_device()
    if len(shape) == 4:
        B, T, Hq, D = shape
    elif len(shape) == 3:
        B, (T, Hq, D) = 1, shape
    else:
        raise ValueError(f"q must be [batch, steps, heads, elements] or [rows, heads, elements], got {shape}")
    rows, Hk = shape[:-2], 0
    if k is not None:
        keyed = tuple(k.shape)
        if len(keyed) != len(shape) or keyed[:-2] != rows or keyed[-1] != D:
            raise ValueError(f"q and k must have the same rows and elements: got {shape} and {keyed}")
        Hk = keyed[-2]
    elif k_weight is not None:
        raise ValueError("k_weight belongs to keys: k is None")
    kinds = _choice(norm, NORMS, "norm"), _choice(pairs, PAIRS, "pairs")
    if not eps >= 0.0:
        raise ValueError(f"eps must be >= 0, got {eps}")
    n = 0
    if frequencies is not None:
        if (frequencies.dtype != torch.float64 or frequencies.dim() != 1 or not frequencies.is_contiguous()
                or frequencies.get_device() != device or frequencies.shape[0] > D // 2):
            raise ValueError(f"frequencies must be a contiguous float64 tensor of at most {D // 2} on {q.device}, got "
                             f"{tuple(frequencies.shape)} {frequencies.dtype} on {frequencies.device}")
        n = frequencies.shape[0]
    apart = 0  # elements between two sequences' positions
    if positions is not None:
        st = positions.stride()
        if (positions.dtype != torch.int32 or positions.shape != rows or positions.get_device() != device
                or (st[-1] != 1 and T > 1)):
            raise ValueError(f"positions must be an int32 tensor {rows} on {q.device} with contiguous steps, got "
                             f"{tuple(positions.shape)} {positions.dtype}, strides {st}, on {positions.device}")
        apart = st[0] if len(st) == 2 else 0
    lens = _ints(lengths, B, q, "lengths")
    sizes = B, T, Hq, Hk, D, n
    head = (*sizes, _sq._types[q.dtype], *kinds, eps, lens, frequencies.data_ptr() if n else 0,
            positions.data_ptr() if positions is not None else 0, apart, *_elements(q, q.shape, q, "q"),
            *(_elements(k, k.shape, q, "k") if k is not None else _NONE), _floats(q_weight, (D,), q, "q_weight"),
            _floats(k_weight, (D,), q, "k_weight"))
    return head, sizes


def _same_type(q, k):
    if k is not None and (k.dtype is not q.dtype or k.get_device() != q.get_device()):
        raise ValueError(f"k must have q's type and device: got {k.dtype} on {k.device}, expected {q.dtype} on {q.device}")


def qk_norm(q, k=None, q_weight=None, k_weight=None, *, norm="rms", eps=1e-6, frequencies=None, positions=None,
            pairs="halves", lengths=None, stream=None):
    """Norms of queries and keys for each head, and a rotation by position, in
    one pass:

        z = x w / n,   n = sqrt(mean(x^2) + eps) ("rms") or sqrt(sum(x^2) + eps) ("l2")
        (y_i, y_j) = (z_i cos f - z_j sin f, z_j cos f + z_i sin f),   f = position frequency[p]

    q: [batch, steps, heads, elements] (or [rows, heads, elements], for a step
    or a packed axis), k (or None) the same with heads of its own; elements
    contiguous, any strides otherwise, at most 512 of them. Weights: float32
    [elements] or None. ``frequencies``: float64 [n], radians a position, n at
    most half the elements: the first 2 n elements are turned, in ``pairs``
    "halves" (p, p + n) or "neighbours" (2 p, 2 p + 1); None: no rotation.
    ``positions``: int32 [batch, steps] (or [rows]) with contiguous steps, as
    one row expanded over the batch has; None: 0, 1, 2, ... along the steps. ``lengths`` (int32 [batch]): rows from lengths[b] on enter no
    sum whatever they hold, and come back zero.

    Returns the normalised q and k (None without), differentiable where an
    input requires a gradient."""
    if stream is not None:
        return _elsewhere(stream, qk_norm, q, k, q_weight, k_weight, norm=norm, eps=eps, frequencies=frequencies,
                          positions=positions, pairs=pairs, lengths=lengths)
    _dtype_of(q, "q")
    _same_type(q, k)
    _no_tangents(q, k, q_weight, k_weight)
    if _wants_grad(q, k, q_weight, k_weight):
        from . import layers

        return layers.qk_norm(q, k, q_weight, k_weight, norm=norm, eps=eps, frequencies=frequencies,
                              positions=positions, pairs=pairs, lengths=lengths)
    head, sizes = _norm_call(q, k, q_weight, k_weight, norm, eps, frequencies, positions, pairs, lengths)
    qy = _empty(q)
    ky = None if k is None else _empty(k)
    if sizes[0] and sizes[1]:
        n = _QK_NORM.pack(*head, *_fresh(qy), *(_NONE if k is None else _fresh(ky)), *_NONE * 4, 0, 0, 0, 0)
        fftmv_qk_norm_forward(n, _current_stream(q.get_device()))
    return qy, ky


def qk_norm_backward(dqy, dky, q, k=None, q_weight=None, k_weight=None, *, norm="rms", eps=1e-6, frequencies=None,
                     positions=None, pairs="halves", lengths=None, stream=None):
    """Gradients of ``qk_norm``: (dq, dk, dq_weight, dk_weight), the last two
    float32 [elements] or None where there is no weight, from those of its
    results. The inputs and keywords are the forward call's."""
    if stream is not None:
        return _elsewhere(stream, qk_norm_backward, dqy, dky, q, k, q_weight, k_weight, norm=norm, eps=eps,
                          frequencies=frequencies, positions=positions, pairs=pairs, lengths=lengths)
    _dtype_of(q, "q")
    _same_type(q, k)
    _no_tangents(dqy, dky, q, k, q_weight, k_weight)
    torch = _sq._torch
    head, sizes = _norm_call(q, k, q_weight, k_weight, norm, eps, frequencies, positions, pairs, lengths)
    if dqy is None or (dky is None) != (k is None):
        raise ValueError("dqy and, with keys, dky must be the gradients of the results: one is missing, or keys are")
    dqf = _elements(dqy, q.shape, q, "dqy")
    dkf = _NONE if k is None else _elements(dky, k.shape, q, "dky")
    dq = _empty(q)
    dk = None if k is None else _empty(k)
    dwq, dwk = (None if w is None else torch.empty_like(w) for w in (q_weight, k_weight))
    if not sizes[0]:
        return dq, dk, *(None if w is None else w.zero_() for w in (dwq, dwk))
    need = _norm_bytes(*sizes[:5]) if dwq is not None or dwk is not None else 0
    ws = q.new_empty(need, dtype=torch.uint8)
    n = _QK_NORM.pack(*head, *_NONE * 2, *dqf, *dkf, *_fresh(dq), *(_NONE if k is None else _fresh(dk)),
                      dwq.data_ptr() if dwq is not None else 0, dwk.data_ptr() if dwk is not None else 0,
                      ws.data_ptr() if need else 0, need)
    fftmv_qk_norm_backward(n, _current_stream(q.get_device()))
    return dq, dk, dwq, dwk
