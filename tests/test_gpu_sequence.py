"""The sequence operators on the GPU against their definitions in float64
(sequence_reference), at the sizes, masks and strides where they can go
wrong. Every output entry is held to a running error bound of float32
arithmetic plus half a unit of its own type."""
import numpy as np
import pytest

import sequence_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def fm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fft_block_toeplitz_amd as fm

    fm.lib()
    return fm


def near(got, want, bound, what):
    got = got.detach().double().cpu().numpy()
    assert got.shape == want.shape, what
    assert np.isfinite(got).all(), f"{what}: not finite"
    worst = np.abs(got - want) - bound
    assert (worst <= 0).all(), f"{what}: {np.abs(got - want).max():.3g} off, {(np.abs(got - want) / bound).max():.3g} bounds"


def fields(seed, shape, dtype, decay, strided=False):
    """x and gate of one type, contiguous or as the halves of one projection (rows 2C + 3 apart)."""
    rng = np.random.default_rng(seed)
    C = shape[-1]
    x = torch.from_numpy(rng.standard_normal(shape)).to(DT[dtype])
    g = rng.standard_normal(shape) * 1.5 + 2.0 + 3.0 * rng.random(C)
    if decay == "value":
        g = 1.0 / (1.0 + np.exp(-g)) * np.where(rng.random(C) < 0.3, -1.0, 1.0)  # some decays alternate
    elif decay == "exp":
        g = -np.log1p(np.exp(-g))
    g = torch.from_numpy(g).to(DT[dtype])
    if not strided:
        return x.cuda(), g.cuda()
    both = torch.full(shape[:-1] + (2 * C + 3,), float("nan"), dtype=DT[dtype], device="cuda")
    both[..., :C] = x.cuda()
    both[..., C:2 * C] = g.cuda()
    return both[..., :C], both[..., C:2 * C]


def host(t):
    return t.detach().double().cpu().numpy()


def check_recurrence(fm, seed, B, T, C, dtype, decay, drive, spans=None, packed=False, strided=False, state=True,
                     dlast=True):
    """Forward and backward of one call. spans: (first, end) of each sequence's steps."""
    shape = (T, C) if packed else (B, T, C)
    x, g = fields(seed, shape, dtype, decay, strided)
    rng = np.random.default_rng(seed + 1000)
    h0 = torch.from_numpy(rng.standard_normal((B, C))).float().cuda() if state else None
    dl = torch.from_numpy(rng.standard_normal((B, C))).float().cuda() if dlast else None
    dh = torch.from_numpy(rng.standard_normal(shape)).to(DT[dtype]).cuda()
    how = {"decay": decay, "drive": drive}
    if packed:
        how["offsets"] = torch.tensor([s[0] for s in spans] + [spans[-1][1]], dtype=torch.int32, device="cuda")
    elif spans is not None:
        how["lengths"] = torch.tensor([e for _, e in spans], dtype=torch.int32, device="cuda")
    spans = spans or [(0, T)] * B
    xv, gv, dv = host(x), host(g), host(dh)
    # values that must not be read: everything that no sequence holds
    hold = np.zeros(shape[:-1], dtype=bool)
    for b, (lo, hi) in enumerate(spans):
        (hold if packed else hold[b])[lo:hi] = True
    off = torch.from_numpy(~hold).cuda()
    x[off], g[off], dh[off] = float("nan"), float("inf"), float("nan")

    h, last, carries = fm.recurrence(x, g, h0, save=True, **how)
    h2, last2 = fm.recurrence(x, g, h0, **how)
    assert torch.equal(h, h2) and torch.equal(last, last2)
    dx, dg, dh0 = fm.recurrence_backward(dh, x, g, carries, h0, dl, **how)
    want = {k: np.zeros(shape) for k in ("h", "dx", "dg", "eh", "edx", "edg")}
    ends = {k: np.zeros((B, C)) for k in ("last", "dh0", "elast", "edh0")}
    for b, (lo, hi) in enumerate(spans):
        pick = (lambda v: v[lo:hi]) if packed else (lambda v: v[b, lo:hi])
        r = R.Recurrence(pick(xv), pick(gv), host(h0)[b] if state else np.zeros(C), decay, drive, dtype, pick(dv),
                         host(dl)[b] if dlast else None)
        for k in want:
            pick(want[k])[:] = getattr(r, k)
        for k in ends:
            ends[k][b] = getattr(r, k)
    near(h, want["h"], want["eh"], "h")
    near(last, ends["last"], ends["elast"], "last state")
    near(dx, want["dx"], want["edx"], "dx")
    near(dg, want["dg"], want["edg"], "dgate")
    near(dh0, ends["dh0"], ends["edh0"], "dh0")


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("decay", ["sigmoid", "exp", "value"])
@pytest.mark.parametrize("drive", ["complement", "plain"])
def test_recurrence_kinds(fm, dtype, decay, drive):
    check_recurrence(fm, 1, 2, 300, 72, dtype, decay, drive)


@pytest.mark.parametrize("B,T,C", [
    (1, 1, 1), (1, 2, 3), (3, 1, 64), (5, 7, 65), (2, 31, 127), (1, 255, 64), (1, 256, 33), (1, 257, 128), (4, 100, 40),
    (1, 1000, 8), (7, 64, 16), (2, 2049, 24), (1, 9000, 5)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_recurrence_sizes(fm, B, T, C, dtype):
    check_recurrence(fm, B * T + C, B, T, C, dtype, "sigmoid", "complement")


@pytest.mark.parametrize("dtype,C", [("fp32", 40), ("bf16", 40), ("bf16", 41), ("fp16", 64)])
def test_recurrence_strided_and_without_states(fm, dtype, C):
    check_recurrence(fm, 5, 3, 270, C, dtype, "sigmoid", "complement", strided=True)
    check_recurrence(fm, 6, 3, 270, C, dtype, "exp", "plain", strided=True, state=False, dlast=False)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lengths", [[0, 300, 1, 299], [0, 0, 0, 0], [300, 300, 300, 300], [256, 255, 257, 44]])
def test_recurrence_padded(fm, dtype, lengths):
    """Rows without a step, full rows, ends at and around a chunk's; what is not held is NaN and infinity."""
    check_recurrence(fm, 7, 4, 300, 48, dtype, "sigmoid", "complement", spans=[(0, n) for n in lengths])


@pytest.mark.parametrize("dtype,C", [("fp32", 36), ("bf16", 64), ("bf16", 37)])
@pytest.mark.parametrize("cuts,T", [([0, 0, 5, 5, 261, 512, 513, 1100, 1100], 1100), ([0, 900], 900),
                                    ([0, 0, 0], 0), ([3, 3, 250, 600], 777), ([0] + list(range(1, 400)), 399),
                                    ([0, 256, 512, 768], 768)])
def test_recurrence_packed(fm, dtype, C, cuts, T):
    """Empty sequences anywhere, ends inside and at a chunk's, many in one chunk, rows of no sequence."""
    check_recurrence(fm, 8, len(cuts) - 1, T, C, dtype, "sigmoid", "complement",
                     spans=list(zip(cuts[:-1], cuts[1:])), packed=True)


def test_recurrence_calls_of_all_shapes_share_a_workspace(fm):
    """Calls whose counters lie where another shape's words were, in turn."""
    shapes = [(1, 3000, 200), (9, 140, 64), (4, 300, 48), (1, 520, 1000), (40, 129, 8), (2, 5000, 16)]
    want = {}
    for turn in range(3):
        for B, T, C in shapes if turn % 2 == 0 else shapes[::-1]:
            for dtype in ("fp32", "bf16"):
                x, g = fields(B + T, (B, T, C), dtype, "sigmoid")
                h, last, carries = fm.recurrence(x, g, save=True)
                grads = fm.recurrence_backward(x, x, g, carries)
                got = [t.clone() for t in (h, last) + grads]
                for a, b in zip(got, want.setdefault((B, T, C, dtype), got)):
                    assert torch.equal(a, b)
                if turn == 0:
                    r = R.Recurrence(host(x)[0], host(g)[0], np.zeros(C), "sigmoid", "complement", dtype, host(x)[0])
                    near(h[0], r.h, r.eh, "h")
                    near(grads[0][0], r.dx, r.edx, "dx")


def test_recurrence_no_steps(fm):
    h0 = torch.randn(3, 5, device="cuda")
    x = torch.empty(3, 0, 5, device="cuda")
    h, last, carries = fm.recurrence(x, x, h0, save=True)
    assert h.shape == (3, 0, 5) and torch.equal(last, h0)
    dx, dg, dh0 = fm.recurrence_backward(x, x, x, carries, h0, 2 * h0)
    assert dx.shape == (3, 0, 5) and torch.equal(dh0, 2 * h0)
    x = torch.empty(0, 4, 5, device="cuda")
    assert fm.recurrence(x, x)[0].shape == (0, 4, 5)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_recurrence_not_finite_stays_in_its_sequence(fm, dtype):
    """An infinity in one sequence of a packed axis makes that channel not
    finite until the sequence ends, and reaches no other sequence, whatever
    chunk it is in; a NaN gate does not vanish."""
    C, cuts = 24, [0, 100, 300, 700, 1500]
    x, g = fields(9, (1500, C), dtype, "sigmoid")
    offs = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    clean, clean_last, carries = fm.recurrence(x, g, offsets=offs, save=True)
    dh = torch.randn(1500, C, device="cuda").to(DT[dtype])
    clean_dx, _, _ = fm.recurrence_backward(dh, x, g, carries, offsets=offs)
    x, g = x.clone(), g.clone()
    x[310, 3], g[120, 7] = float("inf"), float("nan")
    h, last, carries = fm.recurrence(x, g, offsets=offs, save=True)
    dx, dg, _ = fm.recurrence_backward(dh, x, g, carries, offsets=offs)
    bad = torch.zeros(1500, C, dtype=torch.bool, device="cuda")
    bad[310:700, 3], bad[120:300, 7] = True, True
    assert torch.equal(h[~bad], clean[~bad])
    assert not torch.isfinite(h[bad]).any()
    assert torch.isfinite(last).sum() == last.numel() - 2
    assert torch.isnan(dg[120, 7])
    keep = torch.ones(1500, C, dtype=torch.bool, device="cuda")
    keep[100:300, 7] = False
    assert torch.equal(dx[keep], clean_dx[keep])


def test_recurrence_long_memory_and_extreme_gates(fm):
    """Gates of +-200 and decays near one over a long series."""
    T, C = 5000, 16
    x, g = fields(10, (1, T, C), "fp32", "sigmoid")
    g[..., 0], g[..., 1], g[..., 2] = 200.0, -200.0, 9.0
    h, last = fm.recurrence(x, g, torch.ones(1, C, device="cuda"))
    assert torch.equal(h[..., 0], torch.ones(1, T, device="cuda"))  # a = 1, 1 - a = 0 (to 1e-87)
    assert torch.allclose(h[..., 1], x[..., 1], rtol=1e-6, atol=0)
    r = R.Recurrence(host(x)[0], host(g)[0], np.ones(C), "sigmoid", "complement", "fp32")
    near(h[0, :, 2:], r.h[:, 2:], r.eh[:, 2:], "h")


def test_recurrence_is_a_toeplitz_operator_for_constant_decays(fm):
    """With constant decays h = F x with F_k = diag(a^k): the framework's own
    plan, in FP64, gives the same series."""
    Nt, C = 250, 6
    rng = np.random.default_rng(11)
    a = torch.from_numpy(rng.uniform(0.3, 0.99, C)).float().cuda()
    F = torch.diag_embed(a.double()[None] ** torch.arange(Nt, device="cuda")[:, None].double()).contiguous()
    x = torch.from_numpy(rng.standard_normal((Nt, C))).float().cuda()
    plan = fm.Plan(F, fm.FFTMV_ALL_FP64)
    v = plan.apply(x.double().contiguous())
    d = torch.from_numpy(rng.standard_normal((Nt, C))).float().cuda()
    w = plan.apply_adjoint(d.double().contiguous())
    plan.close()
    g = a.expand(Nt, C)
    h, _, carries = fm.recurrence(x, g, decay="value", drive="plain", save=True)
    dx, _, _ = fm.recurrence_backward(d, x, g, carries, decay="value", drive="plain")
    r = R.Recurrence(host(x), host(g), np.zeros(C), "value", "plain", "fp32", host(d))
    near(h, host(v), r.eh + 1e-11 * np.abs(host(v)).max(), "F x")
    near(dx, host(w), r.edx + 1e-11 * np.abs(host(w)).max(), "F* d")


@pytest.mark.parametrize("decay,drive", [("sigmoid", "complement"), ("exp", "plain"), ("value", "complement")])
def test_recurrence_gradient_against_differences(fm, decay, drive):
    """d/de of <h, dh> + <last, dlast> along random directions, by central
    differences of the float32 forward. Rounding: each of the ~100 terms is
    off by at most ~1e-6 of its size, over a step of 2e; truncation: e^2 of
    third derivatives of order one."""
    x, g = fields(12, (2, 9, 5), "fp32", decay)
    rng = np.random.default_rng(13)
    new = lambda *s: torch.from_numpy(rng.standard_normal(s)).float().cuda()  # noqa: E731
    h0, dh, dl = new(2, 5), new(2, 9, 5), new(2, 5)
    _, _, carries = fm.recurrence(x, g, h0, decay=decay, drive=drive, save=True)
    dx, dg, dh0 = fm.recurrence_backward(dh, x, g, carries, h0, dl, decay=decay, drive=drive)

    def value(x, g, h0):
        h, last = fm.recurrence(x, g, h0, decay=decay, drive=drive)
        return float((h.double() * dh).sum() + (last.double() * dl).sum())

    e = 1e-2
    for _ in range(3):
        vx, vg, vh = new(2, 9, 5), new(2, 9, 5), new(2, 5)
        want = (value(x + e * vx, g + e * vg, h0 + e * vh) - value(x - e * vx, g - e * vg, h0 - e * vh)) / (2 * e)
        parts = [dx * vx, dg * vg, dh0 * vh]
        got, size = sum(float(p.double().sum()) for p in parts), sum(float(p.double().abs().sum()) for p in parts)
        assert abs(got - want) <= 100 * 1e-6 * 3 / (2 * e) + 10 * e * e * size


# ------------------------------------------------------------ far offsets
def test_offsets_beyond_32_bits(fm):
    """Rows 2^23 elements apart, the last ones more than 2^31 elements from the first: same bits as side by side."""
    C, far = 20, 1 << 23
    x, g = fields(18, (2, 150, C), "bf16", "sigmoid")
    buffer = torch.empty(300 * far, dtype=torch.bfloat16, device="cuda")
    xs, gs = (buffer[k * 64:].as_strided((2, 150, C), (150 * far, far, 1)) for k in range(2))
    xs.copy_(x)
    gs.copy_(g)
    close, last, carries = fm.recurrence(x, g, save=True)
    h, end, carries_far = fm.recurrence(xs, gs, save=True)
    assert torch.equal(h, close) and torch.equal(end, last) and torch.equal(carries_far, carries)
    want = fm.recurrence_backward(x, x, g, carries)
    assert all(torch.equal(a, b) for a, b in zip(fm.recurrence_backward(xs, xs, gs, carries), want))
    flat = xs.as_strided((300, C), (far, 1))
    assert torch.equal(fm.recurrence_step(flat, gs.as_strided((300, C), (far, 1)), torch.zeros(300, C, device="cuda")),
                       fm.recurrence_step(x.reshape(300, C), g.reshape(300, C), torch.zeros(300, C, device="cuda")))
    w = torch.linspace(0.5, 1.5, C, device="cuda")
    for a, b in ((xs, x), (flat, x.reshape(300, C))):
        y, stats = fm.group_norm(a, 5, w, w, activation="gelu", save=True)
        z, stats_near = fm.group_norm(b, 5, w, w, activation="gelu", save=True)
        assert torch.equal(y, z) and torch.equal(stats, stats_near)
        got = fm.group_norm_backward(a, a, stats, 5, w, w, activation="gelu")
        assert all(torch.equal(p, q) for p, q in zip(got, fm.group_norm_backward(b, b, stats, 5, w, w, activation="gelu")))
    del buffer, xs, gs, flat
    states = torch.empty((1 << 31) + 64, dtype=torch.float32, device="cuda")
    cache = states.as_strided((2, C), (1 << 31, 1))
    cache.zero_()
    out = fm.recurrence_step(x[:, 0], g[:, 0], cache, torch.tensor([1, 0], dtype=torch.int32, device="cuda"))
    zero = torch.zeros(2, C, device="cuda")
    assert torch.equal(out, fm.recurrence_step(x[:, 0], g[:, 0], zero))
    assert torch.equal(cache, zero.flip(0))


# ------------------------------------------------------------------- step
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("B,C", [(1, 1), (3, 65), (4, 500), (33, 264)])
def test_step_against_the_definition(fm, dtype, B, C):
    x, g = fields(B + C, (B, C), dtype, "sigmoid", strided=True)
    rng = np.random.default_rng(14)
    cache = torch.from_numpy(rng.standard_normal((2 * B + 1, C + 5))).float().cuda()
    state = cache[:, :C]  # places further apart than their channels
    old, rest = state.clone(), cache[:, C:].clone()
    slots = torch.from_numpy(rng.permutation(2 * B + 1)[:B].astype(np.int32)).cuda()
    if B > 2:
        slots[1], slots[2] = -1, 2 * B + 1  # idle: below and above the cache
    h = fm.recurrence_step(x, g, state, slots)
    want, bound = host(old), 4 * R.U * np.abs(host(old))
    hw, hb = np.zeros((B, C)), np.full((B, C), 1e-300)
    for b, p in enumerate(slots.tolist()):
        if 0 <= p < 2 * B + 1:
            r = R.Recurrence(host(x)[b:b + 1], host(g)[b:b + 1], host(old)[p], "sigmoid", "complement", dtype)
            want[p], bound[p], hw[b], hb[b] = r.last, r.elast, r.h[0], r.eh[0]
    near(state, want, bound, "state")
    near(h, hw, hb, "h")
    assert torch.equal(cache[:, C:], rest)
    untouched = [p for p in range(2 * B + 1) if p not in slots.tolist()]
    assert torch.equal(state[untouched], old[untouched])


@pytest.mark.parametrize("B,C", [(70001, 3), (70001, 5)])
def test_step_of_many_narrow_streams(fm, B, C):
    """More streams than one grid dimension counts; rows that end inside a vector."""
    x, g = fields(16, (B, C), "fp32", "value")
    state = fields(17, (B, C), "fp32", "value")[0].clone()
    want = host(g) * host(state) + host(x)
    bound = 4 * R.U * (np.abs(host(g) * host(state)) + np.abs(host(x)))
    h = fm.recurrence_step(x, g, state, decay="value", drive="plain")
    near(h, want, bound, "h")
    near(state, want, bound, "state")


@pytest.mark.parametrize("decay,drive", [("sigmoid", "complement"), ("exp", "complement"), ("value", "plain")])
def test_steps_follow_the_whole_series(fm, decay, drive):
    """Step after step gives the series' states, to the reordering of FP32 sums."""
    T, C = 40, 70
    x, g = fields(15, (2, T, C), "fp32", decay)
    h, last = fm.recurrence(x, g, decay=decay, drive=drive)
    state = torch.zeros(2, C, device="cuda")
    outs = [fm.recurrence_step(x[:, t], g[:, t], state, decay=decay, drive=drive) for t in range(T)]
    for b in range(2):
        r = R.Recurrence(host(x)[b], host(g)[b], np.zeros(C), decay, drive, "fp32")
        near(torch.stack([o[b] for o in outs]), r.h, r.eh, "steps")
        near(h[b], r.h, r.eh, "series")
        near(state[b], r.last, r.elast, "state")


# -------------------------------------------------------------- group norm
def check_norm(fm, seed, N, S, G, D, dtype, activation, lengths=None, params=True, strided=False, shift=1.0, ndim=3):
    C = G * D
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((N, S, C)) * (0.5 + rng.random(C)) + shift * rng.standard_normal(C)
    dy = rng.standard_normal((N, S, C))
    x, dy = (torch.from_numpy(v).to(DT[dtype]).cuda() for v in (x, dy))
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(C)).float().cuda() if params else None
    b = torch.from_numpy(0.3 * rng.standard_normal(C)).float().cuda() if params else None
    xv, dv = host(x), host(dy)
    lens = [S] * N if lengths is None else lengths
    for n, m in enumerate(lens):  # what is not held must not be read
        x[n, m:], dy[n, m:] = float("nan"), float("inf")
    if strided:
        wide = torch.full((N, S, C + 7), float("nan"), dtype=DT[dtype], device="cuda")
        wide[..., 3:3 + C] = x
        x = wide[..., 3:3 + C]
    if ndim == 2:
        x, dy = x[:, 0], dy[:, 0]
    elif ndim == 4:
        x, dy = x.reshape(N, -1, 2, C), dy.reshape(N, -1, 2, C)
    how = {"activation": activation,
           "lengths": None if lengths is None else torch.tensor(lens, dtype=torch.int32, device="cuda")}
    y, stats = fm.group_norm(x, G, w, b, eps=1e-5, save=True, **how)
    assert torch.equal(y, fm.group_norm(x, G, w, b, eps=1e-5, **how))
    dx, dw, db = fm.group_norm_backward(dy, x, stats, G, w, b, **how)
    again = fm.group_norm_backward(dy, x, stats, G, w, b, **how)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))
    assert y.shape == x.shape and dx.shape == x.shape
    W = host(w) if params else np.ones(C)
    Bv = host(b) if params else np.zeros(C)
    yw, dxw = np.zeros((N, S, C)), np.zeros((N, S, C))
    ey, edx = np.full((N, S, C), 1e-300), np.full((N, S, C), 1e-300)
    sw, es = np.zeros((N, G, 2)), np.full((N, G, 2), 1e-300)
    dww, dbw, edw, edb = np.zeros(C), np.zeros(C), np.full(C, 1e-300), np.full(C, 1e-300)
    for n, m in enumerate(lens):
        if m:
            r = R.GroupNorm(xv[n, :m], G, W, Bv, 1e-5, activation, dtype, dv[n, :m])
            yw[n, :m], ey[n, :m], dxw[n, :m], edx[n, :m] = r.y, r.ey, r.dx, r.edx
            sw[n, :, 0], sw[n, :, 1], es[n, :, 0], es[n, :, 1] = r.mean, r.rstd, r.emean, r.erstd
            dww, dbw, edw, edb = dww + r.dw, dbw + r.db, edw + r.edw, edb + r.edb
    # the sum over the samples
    edw, edb = edw + R.U * R.DEPTH * np.abs(dww), edb + R.U * R.DEPTH * np.abs(dbw)
    near(stats, sw, es, "stats")
    near(y.reshape(N, S, C), yw, ey, "y")
    near(dx.reshape(N, S, C), dxw, edx, "dx")
    near(dw, dww, edw, "dweight")
    near(db, dbw, edb, "dbias")


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("activation", [None, "silu", "gelu"])
def test_norm_kinds(fm, dtype, activation):
    check_norm(fm, 21, 3, 50, 4, 24, dtype, activation)
    check_norm(fm, 22, 37, 1, 5, 40, dtype, activation, ndim=2)


@pytest.mark.parametrize("N,S,G,D", [
    (1, 1, 1, 2), (2, 1, 3, 25), (1, 3, 1, 1), (2, 7, 33, 3), (1, 130, 2, 64), (3, 64, 1, 500), (1, 1000, 3, 10),
    (2, 2500, 2, 8), (1, 5000, 1, 7), (70, 1, 2, 1000), (300, 1, 4, 32), (2, 4, 64, 2), (1, 2, 1, 4099)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_norm_sizes(fm, N, S, G, D, dtype):
    check_norm(fm, N + S + G + D, N, S, G, D, dtype, "silu")


@pytest.mark.parametrize("N,S,G,D", [
    (2100, 1, 3, 40), (1300, 2, 5, 24), (1205, 1, 2, 25), (1100, 3, 64, 2), (2100, 9, 4, 64), (1, 250, 41, 100),
    (1, 200, 20, 128), (16, 64, 9, 64), (1100, 1, 1, 2056)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_norm_many_samples_and_wide_rows(fm, N, S, G, D, dtype):
    """Sizes that fill the card: several samples a workgroup, whole slabs, and ranges of one sample."""
    check_norm(fm, N + S + G + D, N, S, G, D, dtype, "silu")


def test_norm_many_padded(fm):
    rng = np.random.default_rng(29)
    check_norm(fm, 29, 1500, 4, 3, 40, "bf16", "gelu", lengths=rng.integers(0, 5, 1500).tolist())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_norm_large_mean(fm, dtype):
    """Means of a thousand deviations: the variance is not a difference of squares."""
    check_norm(fm, 23, 2, 300, 4, 16, dtype, None, shift=1000.0 if dtype == "fp32" else 30.0)
    check_norm(fm, 24, 50, 1, 4, 64, dtype, "silu", shift=1000.0 if dtype == "fp32" else 30.0)


@pytest.mark.parametrize("dtype,D", [("fp32", 12), ("bf16", 16), ("bf16", 5)])
@pytest.mark.parametrize("lengths", [[0, 600, 1, 333], [0, 0, 0, 0], [2100, 2100, 0, 2099]])
def test_norm_padded(fm, dtype, D, lengths):
    check_norm(fm, 25, 4, max(max(lengths), 20), 6, D, dtype, "silu", lengths=lengths)


@pytest.mark.parametrize("dtype,D", [("fp32", 8), ("bf16", 16)])
def test_norm_strides_parameters_and_shapes(fm, dtype, D):
    check_norm(fm, 26, 3, 40, 4, D, dtype, "silu", strided=True)
    check_norm(fm, 27, 3, 40, 4, D, dtype, "gelu", params=False)
    check_norm(fm, 28, 3, 40, 4, D, dtype, None, ndim=4)


def test_norm_constant_rows(fm):
    """No variance at all: xhat is 0 and rstd 1/sqrt(eps)."""
    x = torch.full((2, 10, 32), 3.5, device="cuda", dtype=torch.bfloat16)
    y, stats = fm.group_norm(x, 4, save=True)
    assert torch.equal(y, torch.zeros_like(x))
    assert torch.equal(stats[..., 0], torch.full((2, 4), 3.5, device="cuda"))
    assert torch.allclose(stats[..., 1], torch.full((2, 4), 1e5 ** 0.5, device="cuda"), rtol=1e-6)


def test_norm_no_rows(fm):
    x = torch.empty(2, 0, 8, device="cuda")
    y, stats = fm.group_norm(x, 2, save=True)
    assert y.shape == x.shape and torch.equal(stats, torch.zeros(2, 2, 2, device="cuda"))
    dx, dw, db = fm.group_norm_backward(x, x, stats, 2)
    assert torch.equal(dw, torch.zeros(8, device="cuda")) and torch.equal(db, torch.zeros(8, device="cuda"))
    x = torch.empty(0, 3, 8, device="cuda")
    assert fm.group_norm(x, 2).shape == (0, 3, 8)


def test_norm_not_finite_stays_in_its_group(fm):
    x = torch.randn(2, 30, 32, device="cuda")
    clean = fm.group_norm(x, 4, activation="silu")
    x = x.clone()
    x[1, 7, 9] = float("nan")
    y = fm.group_norm(x, 4, activation="silu")
    keep = torch.ones_like(x, dtype=torch.bool)
    keep[1, :, 8:16] = False
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[~keep]).all()


@pytest.mark.parametrize("activation", [None, "silu", "gelu"])
def test_norm_gradient_against_differences(fm, activation):
    """As for the recurrence: ~100 terms, 1e-6 each, steps of 2e."""
    rng = np.random.default_rng(29)
    new = lambda *s: torch.from_numpy(rng.standard_normal(s)).float().cuda()  # noqa: E731
    x, w, b, dy = new(2, 6, 8), new(8), new(8), new(2, 6, 8)
    _, stats = fm.group_norm(x, 2, w, b, activation=activation, save=True)
    dx, dw, db = fm.group_norm_backward(dy, x, stats, 2, w, b, activation=activation)
    value = lambda x, w, b: float((fm.group_norm(x, 2, w, b, activation=activation).double() * dy).sum())  # noqa: E731
    e = 1e-2
    for _ in range(3):
        vx, vw, vb = new(2, 6, 8), new(8), new(8)
        want = (value(x + e * vx, w + e * vw, b + e * vb) - value(x - e * vx, w - e * vw, b - e * vb)) / (2 * e)
        parts = [dx * vx, dw * vw, db * vb]
        got, size = sum(float(p.double().sum()) for p in parts), sum(float(p.double().abs().sum()) for p in parts)
        assert abs(got - want) <= 100 * 1e-6 * 3 / (2 * e) + 10 * e * e * size


# ------------------------------------------------ streams, graphs, outputs
def test_another_stream_and_out(fm):
    x, g = fields(30, (2, 600, 64), "bf16", "sigmoid")
    want, want_last = fm.recurrence(x, g)
    yw = fm.group_norm(want, 4, activation="silu")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out, yo = torch.empty_like(x), torch.empty_like(x)
    side.wait_stream(torch.cuda.current_stream())
    h, last = fm.recurrence(x, g, out=out, stream=side)
    y = fm.group_norm(h, 4, activation="silu", out=yo, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert h is out and y is yo
    assert torch.equal(h, want) and torch.equal(last, want_last) and torch.equal(y, yw)


def test_graph_replays(fm):
    """Forward, backward and step in one graph; every replay gives the eager
    results, with eager calls between the replays."""
    x, g = fields(31, (2, 3000, 72), "bf16", "sigmoid")
    dh = torch.randn(2, 3000, 72, device="cuda").bfloat16()
    w = torch.ones(72, device="cuda")
    state = torch.zeros(2, 72, device="cuda")

    def work():
        h, last, carries = fm.recurrence(x, g, save=True)
        y, stats = fm.group_norm(h, 8, w, activation="silu", save=True)
        dy = fm.group_norm_backward(dh, h, stats, 8, w, activation="silu")
        grads = fm.recurrence_backward(dy[0], x, g, carries)
        one = fm.recurrence_step(x[:, 0], g[:, 0], state)
        return (h, last, y) + dy + grads + (one,)

    eager = [t.clone() for t in work()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for k in range(4):
        state.zero_()
        for t in held:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, eager):
            assert torch.equal(a, b)
        state.zero_()
        again = work()
        torch.cuda.synchronize()
        for a, b in zip(again, eager):
            assert torch.equal(a, b)


def test_two_streams_at_once(fm):
    """Calls on two streams have workspaces of their own."""
    x, g = fields(32, (1, 20000, 128), "bf16", "sigmoid")
    want, want_last = fm.recurrence(x, g)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(4):
        got += [fm.recurrence(x, g, stream=s) for s in (a, b)]
    torch.cuda.synchronize()
    for h, last in got:
        assert torch.equal(h, want) and torch.equal(last, want_last)


# --------------------------------------------------------------- refusals
def test_refusals(fm):
    x = torch.zeros(2, 5, 8, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    bad = [
        lambda: fm.recurrence(x.cpu(), x),
        lambda: fm.recurrence(x.double(), x.double()),
        lambda: fm.recurrence(x, x.bfloat16()),
        lambda: fm.recurrence(x, x[:, :4]),
        lambda: fm.recurrence(x.transpose(1, 2), x.transpose(1, 2)),  # channels not contiguous
        lambda: fm.recurrence(x, x, torch.zeros(2, 7, device="cuda")),
        lambda: fm.recurrence(x, x, torch.zeros(2, 8, device="cuda").bfloat16()),
        lambda: fm.recurrence(x, x, decay="tanh"),
        lambda: fm.recurrence(x, x, drive=None),
        lambda: fm.recurrence(x, x, lengths=i32(1, 2, 3)),
        lambda: fm.recurrence(x, x, lengths=torch.tensor([1, 2], device="cuda")),  # int64
        lambda: fm.recurrence(x, x, offsets=i32(0, 5)),
        lambda: fm.recurrence(x[0], x[0], lengths=i32(5), offsets=i32(0, 5)),
        lambda: fm.recurrence(x, x, out=x),
        lambda: fm.recurrence(x, x, out=x.bfloat16()),
        lambda: fm.recurrence(x[0, 0], x[0, 0]),
        lambda: fm.recurrence_backward(x, x, x, None),
        lambda: fm.recurrence_backward(x, x, x, torch.zeros(2, 8, device="cuda")),
        lambda: fm.recurrence_step(x, x, x[:, 0]),
        lambda: fm.recurrence_step(x[0], x[0], torch.zeros(5, 7, device="cuda")),
        lambda: fm.recurrence_step(x[0], x[0], torch.zeros(4, 8, device="cuda")),
        lambda: fm.recurrence_step(x[0], x[0], torch.zeros(1, 8, device="cuda").expand(5, 8)),
        lambda: fm.recurrence_step(x[0], x[0], torch.zeros(5, 8, device="cuda"), i32(1)),
        lambda: fm.group_norm(x, 3),
        lambda: fm.group_norm(x, 0),
        lambda: fm.group_norm(x, 2, torch.ones(7, device="cuda")),
        lambda: fm.group_norm(x, 2, eps=-1.0),
        lambda: fm.group_norm(x, 2, eps=float("nan")),
        lambda: fm.group_norm(x, 2, activation="relu"),
        lambda: fm.group_norm(x[0, 0], 2),
        lambda: fm.group_norm(x, 2, lengths=i32(1)),
        lambda: fm.group_norm(x.transpose(1, 2), 1),
        lambda: fm.group_norm_backward(x, x, None, 2),
        lambda: fm.group_norm_backward(x[:, :4], x, torch.zeros(2, 2, 2, device="cuda"), 2),
        lambda: fm.group_norm_backward(x, x, torch.zeros(2, 4, 2, device="cuda"), 2),
    ]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"refusal {k} did not raise")
    torch.cuda.synchronize()
