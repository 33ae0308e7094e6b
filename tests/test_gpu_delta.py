"""The gated delta rule and the norms of its queries and keys on the GPU
against their definitions in float64 (delta_reference), at the sizes, masks,
strides and types where they can go wrong."""
import pytest

torch = pytest.importorskip("torch")

import delta_reference as R  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def fm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fft_block_toeplitz_amd as fm

    fm.lib()
    return fm


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def fields(seed, rows, Hk, H, K, V, dtype, decay="sigmoid", rate="sigmoid", strided=False):
    """q, k (unit length), v, gate and beta of one type, contiguous or as parts of one projection."""
    gen, dt = generator(seed), DT[dtype]
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    q, k = (torch.nn.functional.normalize(n(*rows, Hk, K), dim=-1) for _ in range(2))
    v, gate, beta = n(*rows, H, V), n(*rows, H) + 2.0 + 3.0 * torch.rand(H, generator=gen, device="cuda"), n(*rows, H)
    if decay == "exp":
        gate = torch.nn.functional.logsigmoid(gate)
    if rate == "value":
        beta = 2.0 * torch.sigmoid(beta)  # up to 2: 1 - b k k^T still shortens nothing but keeps its norm
    if not strided:
        return [t.to(dt) for t in (q, k, v, gate, beta)]
    sizes = [Hk * K, Hk * K, H * V, H, H]
    p = torch.full((*rows, sum(sizes) + 5), float("nan"), dtype=dt, device="cuda")
    parts = p[..., 3:-2].split(sizes, -1)
    parts = [t.unflatten(-1, (h, w)) for t, h, w in zip(parts, (Hk, Hk, H), (K, K, V))] + list(parts[3:])
    for t, x in zip(parts, (q, k, v, gate, beta)):
        t.copy_(x)
    return parts


def check_delta(fm, seed, B, T, Hk, H, K, V, dtype="bf16", decay="sigmoid", rate="sigmoid", spans=None, packed=False,
                strided=False, state=True, dlast=True, scale=None, change=None):
    """Forward and backward of one call. spans: (first, end) of each sequence's steps."""
    rows = (T,) if packed else (B, T)
    x = fields(seed, rows, Hk, H, K, V, dtype, decay, rate, strided)
    if change:
        change(*x)
    gen = generator(seed + 1000)
    h0 = torch.randn((B, H, K, V), generator=gen, device="cuda") if state else None
    dl = torch.randn((B, H, K, V), generator=gen, device="cuda") if dlast else None
    dy = torch.randn((*rows, H, V), generator=gen, device="cuda").to(DT[dtype])
    how = {"decay": decay, "rate": rate, "scale": scale}
    if packed:
        how["offsets"] = torch.tensor([s[0] for s in spans] + [spans[-1][1]], dtype=torch.int32, device="cuda")
    elif spans is not None:
        how["lengths"] = torch.tensor([e for _, e in spans], dtype=torch.int32, device="cuda")
    spans = spans or [(0, T)] * B
    values = [t.double() for t in x]
    dyv = dy.double()
    hold = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for b, (lo, hi) in enumerate(spans):
        (hold if packed else hold[b])[lo:hi] = True
    for t in (*x, dy):  # values that must not be read
        t[~hold] = float("nan")

    y, last, carries = fm.delta_rule(*x, h0, save=True, **how)
    y2, last2 = fm.delta_rule(*x, h0, **how)
    assert torch.equal(y, y2) and torch.equal(last, last2)
    grads = fm.delta_rule_backward(dy, *x, carries, h0, dl, **how)
    again = fm.delta_rule_backward(dy, *x, carries, h0, dl, **how)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    names = "y dq dk dv dgate dbeta".split()
    for t, name in zip((y, *grads), names):
        assert not t[~hold].any(), f"{name}: rows of no sequence are not zero"
    tol = R.tolerance(DT[dtype])
    for b, (lo, hi) in enumerate(spans):
        pick = (lambda t: t[lo:hi]) if packed else (lambda t: t[b, lo:hi])
        zero = torch.zeros((H, K, V), dtype=torch.float64, device="cuda")
        want = R.delta_rule(*map(pick, values), h0[b].double() if state else zero, decay, rate,
                            K ** -0.5 if scale is None else scale, pick(dyv), dl[b].double() if dlast else None)
        sizes = {"dgate": want[8], "dbeta": want[9]}
        for name, got, ref in zip(names, (y, *grads), (want[0], *want[2:7])):
            if hi > lo:
                for h in range(ref.shape[1]):
                    R.near(pick(got)[:, h], ref[:, h], tol, f"{name}, sequence {b}, head {h}",
                           size_of=sizes[name][:, h] if name in sizes else None)
        for h in range(H):
            R.near(last[b, h], want[1][h], 64 * R.U, f"last state {b}, {h}", rows=False)
            R.near(grads[5][b, h], want[7][h], 64 * R.U, f"dh0 {b}, {h}", rows=False)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("decay", ["sigmoid", "exp"])
@pytest.mark.parametrize("rate", ["sigmoid", "value"])
def test_delta_kinds(fm, dtype, decay, rate):
    check_delta(fm, 1, 2, 150, 2, 2, 64, 64, dtype, decay, rate)


@pytest.mark.parametrize("B,T,Hk,H,K,V", [
    (1, 1, 1, 1, 1, 1), (1, 2, 1, 1, 3, 2), (3, 1, 2, 2, 64, 16), (2, 63, 1, 2, 32, 33), (1, 64, 1, 1, 128, 128),
    (1, 65, 2, 2, 33, 31), (2, 128, 1, 1, 65, 64), (1, 129, 3, 3, 25, 25), (1, 200, 1, 4, 127, 130), (5, 7, 2, 4, 40, 72),
    (1, 500, 1, 1, 128, 200), (1, 300, 1, 2, 96, 17), (33, 3, 2, 2, 8, 8), (1, 70, 1, 1, 16, 1024)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_delta_sizes(fm, B, T, Hk, H, K, V, dtype):
    check_delta(fm, B * T + K + V, B, T, Hk, H, K, V, dtype)


@pytest.mark.parametrize("dtype,K,V", [("fp32", 40, 24), ("bf16", 64, 64), ("bf16", 41, 23), ("fp16", 75, 128)])
def test_delta_strided_and_without_states(fm, dtype, K, V):
    check_delta(fm, 5, 3, 130, 2, 4, K, V, dtype, strided=True)
    check_delta(fm, 6, 3, 130, 1, 3, K, V, dtype, "exp", "value", strided=True, state=False, dlast=False, scale=0.7)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lengths", [[0, 200, 1, 199], [0, 0, 0, 0], [200, 200, 200, 200], [64, 65, 63, 128]])
def test_delta_padded(fm, dtype, lengths):
    """Rows without a step, full rows, ends at and around a run's; what is not held is NaN."""
    check_delta(fm, 7, 4, 200, 2, 2, 48, 40, dtype, spans=[(0, n) for n in lengths])


@pytest.mark.parametrize("dtype,V", [("fp32", 36), ("bf16", 64), ("fp16", 37)])
@pytest.mark.parametrize("cuts,T", [([0, 0, 5, 5, 70, 128, 129, 400, 400], 400), ([0, 300], 300), ([0, 0, 0], 0),
                                    ([3, 3, 130, 260], 333), ([0] + list(range(1, 100)), 99), ([0, 64, 128, 192], 192),
                                    ([60, 70, 71], 500)])
def test_delta_packed(fm, dtype, V, cuts, T):
    """Empty sequences anywhere, ends inside and at a run's, many in one run, rows of no sequence."""
    check_delta(fm, 8, len(cuts) - 1, T, 1, 2, 32, V, dtype, spans=list(zip(cuts[:-1], cuts[1:])), packed=True)


@pytest.mark.parametrize("dtype,B,T,Hk,H,K,V,lengths", [
    ("bf16", 1, 2100, 1, 1, 128, 64, None), ("fp32", 1, 1300, 1, 2, 40, 72, None), ("fp16", 1, 1700, 2, 2, 64, 128, None),
    ("bf16", 3, 1999, 1, 1, 75, 41, None), ("fp32", 4, 1500, 1, 1, 64, 33, [1500, 0, 449, 700]),
    ("bf16", 5, 1536, 1, 1, 32, 16, [1, 1536, 1535, 512, 64]), ("fp32", 1, 1100, 1, 1, 128, 130, None)])
def test_delta_long_sequences_in_parts(fm, dtype, B, T, Hk, H, K, V, lengths):
    """Few heads and many steps: sequences cut into parts, ends inside, at the edges of and in front of parts."""
    check_delta(fm, 13, B, T, Hk, H, K, V, dtype, spans=None if lengths is None else [(0, n) for n in lengths])


def test_delta_parts_keep_what_the_beginning_left(fm):
    """Decays of one: the first part's state reaches the last output."""
    def change(q, k, v, gate, beta):
        gate.fill_(40.0)
        v[:, 64:] = 0.0
        k[:, 64:] = 0.0
        k[:, 64:, :, 0] = 1.0

    check_delta(fm, 14, 1, 1400, 1, 1, 64, 64, "fp32", change=change)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_delta_gates_at_their_ends(fm, dtype):
    """A decay of zero clears the state, one of one keeps it; rates of zero write nothing, of one replace."""
    def change(q, k, v, gate, beta):
        gate[:, 10] = gate[:, 70:75] = float("-inf")
        gate[:, 100:] = 60.0
        beta[:, 20:25] = float("-inf")
        beta[:, 80:85] = 80.0

    check_delta(fm, 9, 2, 150, 2, 2, 32, 32, dtype, change=change)

    def change(q, k, v, gate, beta):
        gate[:, 5] = gate[:, 64] = float("-inf")
        gate[:, 90:] = 0.0
        beta[:, 20:25] = 0.0
        beta[:, 30] = 1e-30
        beta[:, 80:85] = 1.0

    check_delta(fm, 10, 2, 150, 2, 2, 32, 32, dtype, "exp", "value", change=change)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_delta_keys_alike(fm, dtype):
    """The same key at every step: each corrects what the one before has left."""
    def change(q, k, v, gate, beta):
        k.copy_(k[:, :1].expand_as(k))
        beta.fill_(4.0)

    check_delta(fm, 11, 2, 200, 1, 1, 64, 32, dtype, change=change)


def test_delta_is_the_recurrence_with_one_key(fm):
    """With one key that is always one and a rate of one the state is replaced: y_t = scale v_t q_t."""
    q, k, v, gate, beta = fields(12, (2, 100), 1, 1, 1, 24, "fp32", rate="value")
    k.fill_(1.0)
    beta.fill_(1.0)
    y, last = fm.delta_rule(q, k, v, gate, beta, rate="value", scale=0.5)
    torch.testing.assert_close(y, 0.5 * v * q, rtol=2e-6, atol=2e-6)
    torch.testing.assert_close(last[:, 0, 0], v[:, -1, 0], rtol=2e-6, atol=2e-6)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("B,Hk,H,K,V", [(1, 1, 1, 1, 1), (4, 4, 8, 64, 64), (12, 2, 2, 25, 25), (9, 1, 4, 128, 128),
                                        (3, 3, 3, 75, 41), (2, 1, 2, 100, 300), (5, 2, 2, 7, 130)])
def test_delta_step(fm, dtype, B, Hk, H, K, V):
    """Steps against the series, in a cache with more places than streams; idle streams leave it as it is."""
    x = fields(B + K, (B, 5), Hk, H, K, V, dtype, strided=True)
    gen = generator(3)
    places = B + 3
    state = torch.randn((places, H, K, V), generator=gen, device="cuda")
    slots = torch.randperm(places, generator=gen, device="cuda")[:B].to(torch.int32)
    if B > 2:
        slots[1], slots[2] = -1, places
    start = state.clone()
    tol = R.tolerance(DT[dtype])
    want, ys = start.double(), []
    on = (slots >= 0) & (slots < places)
    for t in range(5):
        ys.append(fm.delta_rule_step(*(f[:, t] for f in x), state, slots))
    for b in range(B):
        if not on[b]:
            assert not any(y[b].any() for y in ys)
            continue
        s = int(slots[b])
        y, last = R.delta_rule(*(f[b].double() for f in x), start[s].double(), "sigmoid", "sigmoid", K ** -0.5)
        want[s] = last
        for t in range(5):
            R.near(ys[t][b], y[t], tol, f"y of stream {b}, step {t}", rows=False)
    R.near(state, want, 64 * R.U, "states")
    idle = torch.ones(places, dtype=torch.bool, device="cuda")
    idle[slots[on].long()] = False
    assert torch.equal(state[idle], start[idle])


def check_norm(fm, seed, rows, Hq, Hk, D, dtype, norm, pairs, n, weight, lengths=None, positions=True, strided=False):
    gen, dt = generator(seed), DT[dtype]
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    if strided:
        p = torch.full((*rows, (Hq + Hk) * D + 3), float("nan"), dtype=dt, device="cuda")
        q, k = p[..., 1:1 + Hq * D].unflatten(-1, (Hq, D)), p[..., 1 + Hq * D:1 + (Hq + Hk) * D].unflatten(-1, (Hk, D))
        q.copy_(r(*rows, Hq, D))
        k.copy_(r(*rows, Hk, D))
    else:
        q, k = r(*rows, Hq, D).to(dt), r(*rows, Hk, D).to(dt)
    dq, dk = r(*rows, Hq, D).to(dt), r(*rows, Hk, D).to(dt)
    wq, wk = (1.0 + 0.3 * r(D), 1.0 + 0.3 * r(D)) if weight else (None, None)
    freq = 1000.0 ** (-torch.arange(n, dtype=torch.float64, device="cuda") / n) if n else None
    pos = torch.randint(0, 2 ** 20, rows, generator=gen, device="cuda", dtype=torch.int32) if positions else None
    how = {"norm": norm, "eps": 1e-6, "frequencies": freq, "positions": pos, "pairs": pairs}
    hold = torch.ones(rows, dtype=torch.bool, device="cuda")
    if lengths is not None:
        how["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        hold = torch.arange(rows[-1], device="cuda")[None] < how["lengths"][:, None]
        hold = hold.reshape(rows)
    at = pos if positions else torch.arange(rows[-1], device="cuda").expand(rows)
    for t in (q, k, dq, dk):
        t[~hold] = float("nan")
    qy, ky = fm.qk_norm(q, k, wq, wk, **how)
    gq, gk, gwq, gwk = fm.qk_norm_backward(dq, dk, q, k, wq, wk, **how)
    again = fm.qk_norm_backward(dq, dk, q, k, wq, wk, **how)
    tol = R.tolerance(dt)
    for x, w, d, y, dx, dw, dw2, name in ((q, wq, dq, qy, gq, gwq, again[2], "q"), (k, wk, dk, ky, gk, gwk, again[3], "k")):
        assert not y[~hold].any() and not dx[~hold].any(), name
        ry, rdx, rdw, size = R.qk_norm(x[hold].double(), None if w is None else w.double(), norm, 1e-6, freq, at[hold], pairs,
                                 d[hold].double())
        R.near(y[hold], ry, tol, name)
        R.near(dx[hold], rdx, tol, "d" + name, size_of=size)
        if weight:
            # sums over all rows and heads: up to 100 roundings in line, of either sign; the terms are known to 64 u
            assert torch.equal(dw, dw2)
            most = (d[hold].double().flatten(0, -2).norm(dim=0) ** 2).sum() ** 0.5
            assert (dw.double() - rdw).norm() <= 64 * R.U * most * max(1.0, float(x[hold].double().abs().max())), "dw" + name


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("weight", [True, False])
def test_qk_norm_kinds(fm, dtype, norm, pairs, weight):
    check_norm(fm, 1, (2, 37), 4, 2, 64, dtype, norm, pairs, 32, weight)


@pytest.mark.parametrize("rows,Hq,Hk,D,n", [
    ((1,), 1, 1, 1, 0), ((3,), 2, 1, 2, 1), ((2, 5), 3, 2, 7, 3), ((1, 9), 5, 1, 75, 25), ((4, 1), 8, 8, 64, 32),
    ((1, 100), 3, 3, 128, 10), ((2, 33), 2, 1, 250, 125), ((1, 20), 1, 2, 512, 256), ((1, 20), 1, 1, 511, 200),
    ((1, 3000), 2, 1, 25, 12), ((3, 1000), 1, 1, 128, 64), ((1, 9), 40, 8, 100, 13)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_qk_norm_sizes(fm, rows, Hq, Hk, D, n, dtype, pairs):
    check_norm(fm, D + n, rows, Hq, Hk, D, dtype, "rms", pairs, n, True)


@pytest.mark.parametrize("dtype,D", [("fp32", 64), ("bf16", 64), ("fp16", 75)])
def test_qk_norm_strided_padded_and_default_positions(fm, dtype, D):
    check_norm(fm, 2, (4, 50), 3, 2, D, dtype, "l2", "halves", D // 2, True, lengths=[0, 50, 1, 49], strided=True)
    check_norm(fm, 3, (2, 50), 3, 2, D, dtype, "rms", "neighbours", D // 3, False, positions=False, strided=True)
