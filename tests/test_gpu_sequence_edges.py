"""The sequence operators at the edges of what their entry points accept."""
import math
import threading

import numpy as np
import pytest

import sequence_reference as R
from test_gpu_sequence import check_norm, fields, host, near

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fft_block_toeplitz_amd as fm

    fm.lib()
    return fm


def test_norm_backward_of_no_rows_needs_no_pointer(fm):
    """Without rows every unused pointer may be NULL, the statistics too; the parameters' gradients are zeros."""
    from fft_block_toeplitz_amd import sequence as sq

    N, C, G = 3, 40, 4
    need = sq.fftmv_group_norm_workspace(N, 0, C, G, sq.FFTMV_F32, True)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    dw, db = torch.full((2, C), 7.0, device="cuda")
    sq.fftmv_group_norm_backward(sq._GROUP_NORM.pack(
        N, 0, C, G, sq.FFTMV_F32, 0, 0.0, 0, 0, 0, 0, 0, 0, 0, 0, ws.data_ptr(), need, 0, 0, 0, 0, 0, 0, 0, 0, 0,
        dw.data_ptr(), db.data_ptr()), torch.cuda.current_stream().cuda_stream)
    assert not dw.any() and not db.any()


def test_threads_on_one_stream(fm):
    """Four host threads issue calls of many shapes on the default stream; each gets what it gets alone."""
    shapes = [(1, 3000, 200), (9, 140, 64), (4, 300, 48), (1, 520, 1000), (40, 129, 8), (2, 5000, 16)]
    inputs = [fields(50 + i, s, "bf16", "sigmoid") for i, s in enumerate(shapes)]

    def both(x, g):
        h, last, carries = fm.recurrence(x, g, save=True)
        return (h, last) + fm.recurrence_backward(x, x, g, carries)

    want = [both(*v) for v in inputs]
    torch.cuda.synchronize()
    got, start = [[] for _ in range(4)], threading.Barrier(4)

    def work(k):
        start.wait()
        for i in range(30):
            j = (5 * k + i * (1 + k % 2)) % len(shapes)
            got[k].append((j, both(*inputs[j])))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert sum(map(len, got)) == 120
    for j, outs in sum(got, []):
        assert all(torch.equal(a, b) for a, b in zip(outs, want[j]))


@pytest.mark.parametrize("D", [8185, 8190])
def test_norm_backward_of_the_widest_groups(fm, D):
    """16-bit groups that cut vectors and take all of a workgroup's lanes: the
    backward pass asks for more than 64 KiB of LDS."""
    check_norm(fm, D, 5, 1, 2, D, "bf16", "silu")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,cuts", [(300, [-5, 0, 120, 290, 400, 500]), (300, [-9, -9, 300, 301]), (100, [0, 128, 200]),
                                    (256, [0, 257, 999]), (0, [0, 3, 9])])
def test_recurrence_offsets_are_clamped_as_lengths_are(fm, dtype, T, cuts):
    """Offsets below 0 and above the steps stand for 0 and the steps: sequences
    that end behind the axis end with it, those that start there are empty."""
    C, B = 40, len(cuts) - 1
    x, g = fields(41, (T, C), dtype, "sigmoid")
    h0, dl = torch.randn(2, B, C, device="cuda")
    dh = torch.randn(T, C, device="cuda").to(x.dtype)
    got = []
    for c in (cuts, [min(max(v, 0), T) for v in cuts]):
        # what an output that is not written would be found to hold
        del_me = [torch.full((B, C), float("nan"), device="cuda") for _ in range(4)]
        del del_me
        offs = torch.tensor(c, dtype=torch.int32, device="cuda")
        h, last, carries = fm.recurrence(x, g, h0, offsets=offs, save=True)
        got.append((h, last) + fm.recurrence_backward(dh, x, g, carries, h0, dl, offsets=offs))
    for a, b in zip(*got):
        assert torch.isfinite(b).all() and torch.equal(a, b)


def test_outputs_that_overlap_any_input_are_refused(fm):
    """Not only x and gate: an `out` over states, parameters or index arrays is refused as well."""
    flat = torch.zeros(4096, device="cuda")
    x = torch.zeros(2, 1, 66, device="cuda")
    state, out = flat[:132].view(2, 66), flat[:132].view(2, 1, 66)
    ints = flat.view(torch.int32)
    tokens = torch.zeros(2, 66, device="cuda")
    bad = [
        lambda: fm.recurrence(x, x, state, out=out),
        lambda: fm.recurrence(x, x, out=out, lengths=ints[100:102]),
        lambda: fm.recurrence(x[:, 0], x[:, 0], out=out[:, 0], offsets=ints[:4]),
        lambda: fm.recurrence_step(tokens, tokens, torch.zeros(2, 66, device="cuda"), ints[4:6], out=out[:, 0]),
        lambda: fm.recurrence_step(tokens, tokens, state, out=out[:, 0]),
        lambda: fm.group_norm(tokens, 2, weight=flat[:66], out=out[:, 0]),
        lambda: fm.group_norm(tokens, 2, bias=flat[66:132], out=out[:, 0]),
        lambda: fm.group_norm(x, 2, lengths=ints[131:133], out=out),
    ]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError, match="overlap"):
            call()
            pytest.fail(f"refusal {k} did not raise")
    # side by side is no overlap
    assert fm.recurrence(x, x, flat[132:264].view(2, 66), out=out)[0] is out


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("decay,drive", [("value", "plain"), ("exp", "plain"), ("value", "complement")])
@pytest.mark.parametrize("bits,steps", [(2, 100), (10, 20)])
def test_recurrence_of_decays_above_one(fm, dtype, decay, drive, bits, steps):
    """Growth by 2^200 in a window of some steps, which no FP32 product of
    decays holds, over states and gradients that are zero or 2^-110: what the
    definition gives is in range, and so is what the kernels give."""
    B, T, C = 3, 700, 72
    x, g = fields(42, (B, T, C), dtype, decay)
    dh, dl = torch.randn(B, T, C, device="cuda").to(x.dtype), torch.randn(B, C, device="cuda")
    of = (lambda a: a) if decay == "value" else lambda a: float(np.log(a))  # noqa: E731
    small = 2.0 ** -110
    for b, t in enumerate((60, 128, 301)):  # over a chunk's edge, inside one, over a later edge
        end = t + steps
        x[b, :end] = 0.0
        g[b, :t], g[b, t:end], g[b, end:] = of(1.0), of(2.0 ** bits), of(0.5)
        dh[b, t:end] = 0.0
        dh[b, end:] *= small
    dl *= small
    dh[..., 1::3] = 0.0
    dl[:, 1::3] = 0.0
    h0 = torch.zeros(B, C, device="cuda")
    h0[:, ::3] = small
    for lengths in (None, [700, 500, 300]):
        lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
        how = {"decay": decay, "drive": drive, "lengths": lens}
        h, last, carries = fm.recurrence(x, g, h0, save=True, **how)
        dx, dg, dh0 = fm.recurrence_backward(dh, x, g, carries, h0, dl, **how)
        for b in range(B):
            n = T if lengths is None else lengths[b]
            r = R.Recurrence(host(x)[b, :n], host(g)[b, :n], host(h0)[b], decay, drive, dtype, host(dh)[b, :n], host(dl)[b])
            assert max(np.abs(v).max() for v in (r.h, r.dx, r.dg, r.dh0)) < 1e38  # the definition is in range
            for got, want, bound, what in ((h[b, :n], r.h, r.eh, "h"), (last[b], r.last, r.elast, "last state"),
                                           (dx[b, :n], r.dx, r.edx, "dx"), (dg[b, :n], r.dg, r.edg, "dgate"),
                                           (dh0[b], r.dh0, r.edh0, "dh0")):
                near(got, want, bound + 2.0 ** -126, what)  # the smallest normal number


def _candidates(g):
    """(a, 1 - a, da/dg) of a sigmoid in FP32, correctly rounded but for the
    exponential, which may be one unit in the last place off: all that can come out."""
    f = np.float32
    true = np.exp(-np.abs(g.astype(np.float64)))
    t = true.astype(f)
    for t in (t, np.nextafter(t, f(0)), np.nextafter(t, f(np.inf))):
        big = f(1) / (f(1) + t)
        small = t * big
        yield np.where(g >= 0, big, small), np.where(g >= 0, small, big), big * small


def test_fp32_decays_are_rounded_once_an_operation(fm):
    """One step from a state of one (the decay), with a drive of one (its
    complement), and their gradient by the gate (the slope)."""
    rng = np.random.default_rng(43)
    C = 20000
    gv = rng.uniform(-12, 12, C).astype(np.float32)
    g = torch.from_numpy(gv).cuda().view(1, 1, C)
    zero, one = torch.zeros(1, 1, C, device="cuda"), torch.ones(1, 1, C, device="cuda")
    a, _, carries = fm.recurrence(zero, g, one[0], drive="plain", save=True)
    _, slope, _ = fm.recurrence_backward(one, zero, g, carries, one[0], drive="plain")
    rest, _ = fm.recurrence(one, g)
    step_a = fm.recurrence_step(zero[0], g[0], torch.ones(1, C, device="cuda"), drive="plain")
    step_rest = fm.recurrence_step(one[0], g[0], torch.zeros(1, C, device="cuda"))
    may = list(_candidates(gv))
    for got, k, what in ((a, 0, "a"), (rest, 1, "1 - a"), (slope, 2, "slope"), (step_a, 0, "step's a"),
                         (step_rest, 1, "step's 1 - a")):
        got = got.flatten().cpu().numpy()
        assert np.any([got == m[k] for m in may], axis=0).all(), what


def _values_and_slopes(fm, activation, z):
    """act(z) and act'(z) by themselves: groups of (1, -1) have mean 0 and
    deviation 1, a weight of zero leaves z to the bias."""
    C = z.size
    x = torch.tensor([1.0, -1.0], device="cuda").repeat(C // 2).view(1, C)
    b, w = torch.from_numpy(z).cuda(), torch.zeros(C, device="cuda")
    y, stats = fm.group_norm(x, C // 2, w, b, eps=0.0, activation=activation, save=True)
    assert torch.equal(stats, torch.tensor([0.0, 1.0], device="cuda").expand_as(stats))
    _, _, db = fm.group_norm_backward(torch.ones_like(x), x, stats, C // 2, w, b, activation=activation)
    return host(y)[0], host(db)


def _points(far):
    rng = np.random.default_rng(44)
    z = np.concatenate([rng.standard_normal(8000), rng.uniform(-far, far, 8000), [0.0, -0.0, 1e-30, -1e-30]])
    return z.astype(np.float32)


def test_fp32_silu_to_a_few_roundings(fm):
    """With e = exp(-z) (3 U: an ulp and a rounding), 1 + e (U, and e's share of
    its error), the quotient (U) the sigmoid p is off by 5 U, y by 6 U. The slope
    is p + (p z) q: where z > 2 q = e p is off by its factors' 8 U and a rounding,
    of which 1 + e takes back what it grows by, else q = 1 - p by p's error, which
    so enters the slope by its derivative 1 + z (1 - 2 p) alone, under 1 for z > -1
    and under |z| below. Products and sum 3 U: together 12 U of p |z| q and 7 U of
    the slope."""
    z = _points(80.0)
    y, s = _values_and_slopes(fm, "silu", z)
    v = z.astype(np.float64)
    p, q = 1.0 / (1.0 + np.exp(-v)), 1.0 / (1.0 + np.exp(v))
    want, slope = v * p, p * (1.0 + v * q)
    assert (np.abs(y - want) <= 6 * R.U * np.abs(want)).all(), np.nanmax(np.abs(y - want) / np.abs(want)) / R.U
    bound = R.U * (12 * p * np.abs(v) * q + 7 * np.abs(slope))
    assert (np.abs(s - slope) <= bound).all(), (np.abs(s - slope) / bound).max()


def test_fp32_gelu_to_a_few_roundings(fm):
    """Phi = exp(-z^2/2) t R(t) / 2: the exponential 3 U, its exponent's remainder
    and what takes it in 2 U; t from its argument and the quotient 2 U, by which t
    R(t) changes 2.4 times as much; R's fit 2 U, coefficients and sums 3 U; three
    products: 17 U of Phi. Near zero 1/2 + z P less than that. y = z Phi: 18 U. The
    slope Phi + z phi(z): 17 U of Phi, and of the second term the bell's 5 U,
    constant and products 3 U, the sum's rounding of either U."""
    z = _points(12.0)
    y, s = _values_and_slopes(fm, "gelu", z)
    v = z.astype(np.float64)
    phi = 0.5 * np.vectorize(math.erfc)(-v / math.sqrt(2.0))
    second = v * np.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    assert (np.abs(y - v * phi) <= 18 * R.U * np.abs(v * phi)).all(), np.nanmax(np.abs(y / (v * phi) - 1)) / R.U
    bound = R.U * (18 * phi + 9 * np.abs(second))
    assert (np.abs(s - phi - second) <= bound).all(), (np.abs(s - phi - second) / bound).max()


# FP32 numbers whose sum, one after the other, drifts: each addition rounds the same way over a whole binade. Their
# sum over 512, 1024 terms is off by 128 and 256 U.
DRIFTS = {512: 1.0118866, 1024: 1.9810181, 4096: 1.9963379, 16384: 1.9794922}


def test_norm_parameter_gradients_of_many_tokens(fm):
    """65536 tokens whose dy is the same drifting number: dbias is a product."""
    N, G, D = 65536, 16, 1028
    x = torch.randn(1, G * D, device="cuda")
    y, stats = fm.group_norm(x, G, save=True)
    dy = torch.full((1, G * D), DRIFTS[1024], device="cuda")
    _, _, db = fm.group_norm_backward(dy.expand(N, -1), x.expand(N, -1), stats.expand(N, -1, -1).contiguous(), G)
    want = np.full(G * D, N * float(np.float32(DRIFTS[1024])))
    near(db, want, R.U * R.DEPTH * want, "dbias")


def check_constant_gradient(fm, N, S, C, G):
    """x at its mean and dy one drifting number c: dbias is a product, and dx what the mean of dy is off from c."""
    x = torch.ones(1, 1, C, device="cuda").expand(N, S, C)
    dy = torch.full((1, 1, C), DRIFTS[512], device="cuda").expand(N, S, C)
    dx, dw, db = fm.group_norm_backward(dy, x, torch.ones(N, G, 2, device="cuda"), G)
    c = float(np.float32(DRIFTS[512]))
    near(db, np.full(C, N * S * c), np.full(C, R.U * R.DEPTH * N * S * c), "dbias")
    assert not dw.any()
    near(dx[::512], np.zeros(dx[::512].shape), np.full((1, 1, 1), (R.DEPTH + 4.0) * R.U * c), "dx")


def test_norm_sums_of_many_rows_by_few_threads(fm):
    """As many samples as fill the card, each 16384 rows in one range: their
    variance, and the sums of the backward pass, from rows that all add the same
    drifting number."""
    N, S, C = 1025, 16384, 128
    sign = 1.0 - 2.0 * (torch.arange(S, device="cuda") // 8 % 2)
    v = float(np.sqrt(np.float32(DRIFTS[512])))
    x = (sign[:, None] * v).expand(S, C).contiguous()[None]
    y, stats = fm.group_norm(x.expand(N, -1, -1), 1, save=True, eps=0.0)
    vf = float(np.float32(v))
    near(stats[::64, 0, 0], np.zeros(17), np.full(17, R.U * R.DEPTH * vf), "mean")
    # the variance's own sum is off by DEPTH U at most, its root by half of that
    near(stats[::64, 0, 1], np.full(17, 1.0 / vf), np.full(17, (0.5 * R.DEPTH + 4.0) * R.U / vf), "rstd")
    del y
    check_constant_gradient(fm, N, S, C, 1)


def test_norm_joins_many_ranges(fm):
    """One sample of 65536 rows in a thousand ranges, 256 groups of one
    channel: few threads a group to join them."""
    S, C = 65536, 256
    sign = 1.0 - 2.0 * (torch.arange(S, device="cuda") // 8 % 2)
    v = float(np.sqrt(np.float32(DRIFTS[512])))
    x = (sign[:, None] * v).expand(S, C).contiguous()[None]
    _, stats = fm.group_norm(x, C, save=True, eps=0.0)
    vf = float(np.float32(v))
    near(stats[0, :, 1], np.full(C, 1.0 / vf), np.full(C, (0.5 * R.DEPTH + 4.0) * R.U / vf), "rstd")
    check_constant_gradient(fm, 1, S, C, C)


def test_norm_wide_groups_of_many_rows(fm):
    """Groups wider than a workgroup, 4096 rows of one drifting number."""
    S, D = 4096, 4100
    x = torch.full((1, 1, D), DRIFTS[4096], device="cuda").expand(1, S, D)
    c = float(np.float32(DRIFTS[4096]))
    _, stats = fm.group_norm(x, 1, save=True)
    near(stats[0, 0, :1], np.full(1, c), np.full(1, R.U * R.DEPTH * c), "mean")
    S = 16384
    x = torch.randn(1, 1, D, device="cuda")
    _, stats = fm.group_norm(x, 1, save=True)
    dy = torch.full((1, 1, D), DRIFTS[512], device="cuda").expand(1, S, D)
    _, _, db = fm.group_norm_backward(dy, x.expand(1, S, D), stats, 1)
    want = np.full(D, S * float(np.float32(DRIFTS[512])))
    near(db, want, R.U * R.DEPTH * want, "dbias")


@pytest.mark.parametrize("N,S,G,D,dtype,lengths", [
    (3, 5, 2, 4100, "fp32", [5, 0, 3]), (2, 70, 1, 4099, "fp32", None), (2, 40, 3, 8200, "bf16", [40, 33]),
    (5, 1, 1, 9001, "fp16", None), (1, 65, 2, 8193, "bf16", None)])
def test_norm_wide_groups(fm, N, S, G, D, dtype, lengths):
    check_norm(fm, 45, N, S, G, D, dtype, "silu", lengths=lengths)


@pytest.mark.parametrize("N,S,G,D,dtype,lengths", [
    (300, 1, 1, 8200, "bf16", None), (100, 1, 3, 4100, "fp32", None), (520, 2, 2, 4097, "fp32", None),
    (2, 300, 1, 16389, "bf16", [300, 11]), (1, 33, 2, 12290, "fp32", None), (3, 3, 1, 5121, "fp32", [0, 3, 1]),
    (1, 1, 1, 40001, "fp16", None), (1, 700, 2, 8193, "fp16", None)])
def test_norm_wide_groups_in_pieces_and_whole(fm, N, S, G, D, dtype, lengths):
    """Groups wider than a workgroup's lanes: one workgroup each for a row or
    two of many samples, else cut into pieces; last pieces of few channels and
    of whole ones, several groups, padded samples."""
    check_norm(fm, 46, N, S, G, D, dtype, "gelu", lengths=lengths)


def test_norm_wide_groups_without_rows(fm):
    x = torch.empty(3, 0, 9000, device="cuda")
    y, stats = fm.group_norm(x, 1, save=True)
    assert y.shape == x.shape and not stats.any()
    _, dw, db = fm.group_norm_backward(x, x, stats, 1)
    assert not dw.any() and not db.any()


def test_norm_wide_groups_take_no_longer_than_others(fm):
    """4000 rows of 5000 FP32 channels, as one group and as five: within ten
    times of one another (one workgroup for all rows took a thousand times)."""
    x = torch.randn(1, 4000, 5000, device="cuda")
    times = []
    for groups in (5, 1):
        def work():
            _, stats = fm.group_norm(x, groups, save=True)
            fm.group_norm_backward(x, x, stats, groups)

        work()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(3):
            work()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    assert times[1] < 10 * times[0]
