"""Autograd through the gated delta rule and the queries' and keys' norms, the
layer made of them, and the calls that the torch forms take and refuse."""
import pytest

torch = pytest.importorskip("torch")

import delta_reference as R  # noqa: E402
from test_gpu_delta import DT, fields, generator  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fft_block_toeplitz_amd as fm

    fm.lib()
    return fm


def test_gradients_are_the_backward_calls(fm):
    """delta_rule and qk_norm of leaves one after the other: the same numbers as by hand."""
    gen = generator(1)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    leaves = [n(2, 90, 2, 32), n(2, 90, 2, 32), 1 + 0.1 * n(32), 1 + 0.1 * n(32), n(2, 90, 4, 24), n(2, 90, 4), n(2, 90, 4),
              n(2, 4, 32, 24)]
    for t in leaves:
        t.requires_grad_()
    q0, k0, wq, wk, v, gate, beta, h0 = leaves
    freq = 100.0 ** (-torch.arange(16, dtype=torch.float64, device="cuda") / 16)
    lengths = torch.tensor([90, 50], dtype=torch.int32, device="cuda")
    q, k = fm.qk_norm(q0, k0, wq, wk, norm="l2", frequencies=freq, lengths=lengths)
    y, last = fm.delta_rule(q, k, v, gate, beta, h0, lengths=lengths)
    dy, dl = n(2, 90, 4, 24), n(2, 4, 32, 24)
    grads = torch.autograd.grad((y, last), leaves, (dy, dl))
    with torch.no_grad():
        how = {"norm": "l2", "frequencies": freq, "lengths": lengths}
        q, k = fm.qk_norm(q0, k0, wq, wk, **how)
        y2, last2, carries = fm.delta_rule(q, k, v, gate, beta, h0, lengths=lengths, save=True)
        dq, dk, dv, dg, db, dh0 = fm.delta_rule_backward(dy, q, k, v, gate, beta, carries, h0, dl, lengths=lengths)
        dq0, dk0, dwq, dwk = fm.qk_norm_backward(dq, dk, q0, k0, wq, wk, **how)
    assert torch.equal(y, y2) and torch.equal(last, last2)
    for got, want in zip(grads, (dq0, dk0, dwq, dwk, dv, dg, db, dh0)):
        assert torch.equal(got, want)


def test_gradients_against_differences(fm):
    """Along one direction for all inputs at once, in float32: a central difference of step 2^-8 is off by a third
    derivative's 2^-16 / 6 of the derivative's own size, and by the loss's roundings (64 u of its terms' norm) over
    the step."""
    x = fields(2, (1, 80), 2, 4, 16, 12, "fp32")
    gen = generator(3)
    h0 = torch.randn((1, 4, 16, 12), generator=gen, device="cuda")
    wy, wl = (torch.randn(s, generator=gen, device="cuda") for s in ((1, 80, 4, 12), (1, 4, 16, 12)))
    leaves = [t.clone().requires_grad_() for t in (*x, h0)]

    def loss(ts):
        q, k = fm.qk_norm(ts[0], ts[1], norm="l2", positions=None)
        y, last = fm.delta_rule(q, k, *ts[2:])
        return (y.double() * wy).sum() + (last.double() * wl).sum(), (y.norm() * wy.norm() + last.norm() * wl.norm())

    value, _ = loss(leaves)
    grads = torch.autograd.grad(value, leaves)
    for i, leaf in enumerate(leaves):
        d = torch.randn(leaf.shape, generator=gen, device="cuda")
        d = d * (leaf.norm() / d.norm())
        step = 2.0 ** -8
        with torch.no_grad():
            moved = [[t + (s * step * d if j == i else 0.0) for j, t in enumerate(leaves)] for s in (1.0, -1.0)]
            (up, size), (down, _) = loss(moved[0]), loss(moved[1])
        slope, want = float((grads[i].detach().double() * d).sum().detach()), float(up - down) / (2 * step)
        off = float(grads[i].norm() * d.norm()) * 2.0 ** -14 + 64 * R.U * float(size) / step
        assert abs(slope - want) <= off, (i, slope, want, off)


def test_one_output_alone_and_reordered_gradients(fm):
    x = [t.requires_grad_() for t in fields(4, (2, 70), 1, 2, 16, 16, "bf16")]
    y, last = fm.delta_rule(*x)
    a = torch.autograd.grad(last.sum(), x, retain_graph=True)
    b = torch.autograd.grad(y.float().transpose(1, 2).sum(), x, retain_graph=True)
    c = torch.autograd.grad(y.float().sum() + last.sum(), x)
    for s, t, u in zip(a, b, c):
        assert torch.isfinite(s).all() and torch.isfinite(t).all()
        R.near(u, s.double() + t.double(), 3 * R.tolerance(torch.bfloat16), "sum of gradients", rows=False,
               size_of=s.double().abs() + t.double().abs())
    q = torch.randn((3, 5, 2, 24), device="cuda", requires_grad=True)
    qy, ky = fm.qk_norm(q)
    assert ky is None
    qy.sum().backward()
    assert q.grad.shape == q.shape


def test_layer_streams_what_it_says_of_series(fm):
    from fft_block_toeplitz_amd.layers import DeltaLayer

    for dtype, base, key_heads in ((torch.float32, None, 4), (torch.float32, 100.0, 2), (torch.bfloat16, 100.0, 2)):
        torch.manual_seed(0)
        layer = DeltaLayer(10, 4, 16, 24, 6, key_heads=key_heads, base=base).to(dtype)
        x = torch.randn((3, 75, 10), device="cuda", dtype=dtype)
        lengths = torch.tensor([75, 40, 0], dtype=torch.int32, device="cuda")
        with torch.no_grad():
            whole, last = layer(x)
            _, cut = layer(x, lengths=lengths)
            state = torch.zeros((5, 4, 16, 24), device="cuda")
            slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
            streamed = []
            for t in range(75):
                at = torch.full((3,), t, dtype=torch.int32, device="cuda")
                streamed.append(layer.step(x[:, t], state, slots, at if base else None))
                if t == 39:
                    short = state[0].clone()
        # the series takes 64 steps at once, so q, k and y are rounded alike and the states differ by FP32 roundings;
        # y's own rounding may fall to either side, and the linear layer behind adds its own
        tol = 64 * R.U if dtype is torch.float32 else 4 * R.HALF[dtype]
        R.near(torch.stack(streamed, 1), whole.double(), 4 * tol, "streamed")
        R.near(state[slots.long()], last.double(), 64 * R.U, "states")
        R.near(short, cut[1].double(), 64 * R.U, "state of a shorter series", rows=False)
        assert not cut[2].any()
        loss = layer(x)[0].float().square().mean()
        loss.backward()
        assert all(p.grad is not None and torch.isfinite(p.grad).all() for p in layer.parameters())


def test_layer_refuses(fm):
    from fft_block_toeplitz_amd.layers import DeltaLayer

    with pytest.raises(ValueError):
        DeltaLayer(4, 3, 8, 8, 4, key_heads=2)
    layer = DeltaLayer(4, 2, 8, 8, 4, base=10.0)
    with pytest.raises(ValueError):
        layer.step(torch.randn((2, 4), device="cuda"), torch.zeros((2, 2, 8, 8), device="cuda"))


def test_surrogate_with_a_delta_layer(fm):
    from fft_block_toeplitz_amd import surrogate

    result = surrogate.run(iterations=4, Nt=70, batch=4, channels=32, report=None, layer="delta")
    assert result["stream_against_series"] < 1e-4 and result["state_against_series"] < 1e-4
    with pytest.raises(ValueError):
        surrogate.run(layer="other")


def test_refusals(fm):
    q, k, v, gate, beta = fields(5, (2, 10), 2, 4, 16, 8, "bf16")
    good = dict(q=q, k=k, v=v, gate=gate, beta=beta)
    state = torch.zeros((2, 4, 16, 8), device="cuda")
    bad = [dict(q=q.float()), dict(k=k[:, :, :1]), dict(v=v[:1]), dict(v=v[:, :, :3]), dict(gate=gate[..., :2]),
           dict(beta=beta.float()), dict(q=q.transpose(2, 3).contiguous().transpose(2, 3)), dict(v=v.cpu()),
           dict(h0=state[:1]), dict(h0=state.bfloat16()), dict(decay="value"), dict(rate="exp"),
           dict(lengths=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(out=v), dict(out=torch.empty_like(v).float()),
           dict(lengths=torch.zeros(2, dtype=torch.int32, device="cuda"),
                offsets=torch.zeros(2, dtype=torch.int32, device="cuda")),
           dict(offsets=torch.zeros(2, dtype=torch.int32, device="cuda"))]
    for change in bad:
        with pytest.raises(ValueError):
            fm.delta_rule(**{**good, **change})
    wide = torch.zeros((2, 10, 2, 129), device="cuda", dtype=torch.bfloat16)
    with pytest.raises(fm.FftmvError) as e:
        fm.delta_rule(wide, wide, v, gate, beta)
    assert e.value.status == fm.FFTMV_ERR_UNSUPPORTED_SIZE
    y, last, carries = fm.delta_rule(*good.values(), save=True)
    for change in (dict(dy=y[:1]), dict(dy=y.float()), dict(carries=None), dict(carries=carries[:1]),
                   dict(dh_last=state[:1])):
        with pytest.raises(ValueError):
            fm.delta_rule_backward(**{**good, "dy": y, "carries": carries, **change})
    step = {n: t[:, 0] for n, t in good.items()}
    for change in (dict(state=state[:1]), dict(state=state.double()), dict(state=state[:, :3]),
                   dict(state=state.transpose(2, 3).contiguous().transpose(2, 3)), dict(q=q),
                   dict(slots=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(out=step["v"])):
        with pytest.raises(ValueError):
            fm.delta_rule_step(**{**step, "state": state, **change})
    with pytest.raises(ValueError):
        fm.delta_rule_step(**{**step, "v": step["v"].clone().requires_grad_()}, state=state)
    with pytest.raises(ValueError):
        fm.delta_rule(q, k, v.clone().requires_grad_(), gate, beta, out=torch.empty_like(v))
    freq = torch.ones(8, dtype=torch.float64, device="cuda")
    pos = torch.zeros((2, 10), dtype=torch.int32, device="cuda")
    for change in (dict(k=k.float()), dict(k=k[:, :5]), dict(norm="l1"), dict(pairs="odd"), dict(eps=-1.0),
                   dict(frequencies=freq.float()), dict(frequencies=torch.ones(9, dtype=torch.float64, device="cuda")),
                   dict(positions=pos.long()), dict(positions=pos[:1]), dict(q_weight=torch.ones(8, device="cuda")),
                   dict(k=None, k_weight=torch.ones(16, device="cuda"))):
        with pytest.raises(ValueError):
            fm.qk_norm(**{"q": q, "k": k, "frequencies": freq, "positions": pos, **change})
    assert DT["bf16"] is q.dtype


def test_empty_calls(fm):
    q, k, v, gate, beta = (t[:0] for t in fields(6, (2, 10), 2, 4, 16, 8, "bf16"))
    y, last, carries = fm.delta_rule(q, k, v, gate, beta, save=True)
    assert y.shape == v.shape and last.shape == (0, 4, 16, 8)
    assert [t.shape for t in fm.delta_rule_backward(y, q, k, v, gate, beta, carries)][:5] == [
        t.shape for t in (q, k, v, gate, beta)]
    q, k, v, gate, beta = (t[:, :0] for t in fields(6, (2, 10), 2, 4, 16, 8, "bf16"))
    h0 = torch.randn((2, 4, 16, 8), device="cuda")
    y, last, carries = fm.delta_rule(q, k, v, gate, beta, h0, save=True)
    assert torch.equal(last, h0)
    assert torch.equal(fm.delta_rule_backward(y, q, k, v, gate, beta, carries, h0, h0)[5], h0)
    w = torch.ones(16, device="cuda")
    qy, ky = fm.qk_norm(q, k, w, w)
    assert qy.shape == q.shape and ky.shape == k.shape
    grads = fm.qk_norm_backward(qy, ky, q, k, w, w)
    assert not grads[2].any() and not grads[3].any()


def test_graph_replays_and_other_streams(fm):
    """Captured once, replayed on new inputs, with eager calls and another graph's between; a call on another stream."""
    x = fields(7, (2, 130), 2, 4, 32, 32, "bf16")
    w = torch.ones(32, device="cuda")
    gen = generator(8)
    dy = torch.randn((2, 130, 4, 32), generator=gen, device="cuda").bfloat16()

    def work(q, k, v, gate, beta):
        qn, kn = fm.qk_norm(q, k, w, w, norm="l2")
        y, last, carries = fm.delta_rule(qn, kn, v, gate, beta, save=True)
        grads = fm.delta_rule_backward(dy, qn, kn, v, gate, beta, carries)
        return (y, last, *grads, *fm.qk_norm_backward(grads[0], grads[1], q, k, w, w, norm="l2"))

    work(*x)
    graphs = []
    for _ in range(2):
        held = [t.clone() for t in x]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = work(*held)
        graphs.append((graph, held, out))
    for seed in range(4):
        new = fields(20 + seed, (2, 130), 2, 4, 32, 32, "bf16")
        want = [t.clone() for t in work(*new)]
        graph, held, out = graphs[seed % 2]
        for t, u in zip(held, new):
            t.copy_(u)
        graph.replay()
        work(*x)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    side = torch.cuda.Stream()
    want = fm.delta_rule(*x)
    side.wait_stream(torch.cuda.current_stream())
    got = fm.delta_rule(*x, stream=side)
    qs = fm.qk_norm(x[0], x[1], w, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(qs[0], fm.qk_norm(x[0], x[1], w, w)[0])


def test_written_states_raise_version_counters(fm):
    x = [t[:, 0] for t in fields(9, (2, 1), 1, 1, 8, 8, "fp32")]
    state = torch.zeros((2, 1, 8, 8), device="cuda")
    before = state._version
    fm.delta_rule_step(*x, state)
    assert state._version > before
