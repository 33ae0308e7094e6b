"""The differentiable forms against automatic differentiation of the plain
formulas in float64, the layer step by step against the whole series, and the
operators together in the surrogate example."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fft_block_toeplitz_amd as fm

    fm.lib()
    return fm


def leaf(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").requires_grad_()


def off(x, ref):
    return float((x.detach().double() - ref).norm() / ref.norm())


def test_gradients_through_both_operators(fm):
    """One loss through the recurrence (strided halves of a projection, last
    states included) and the normalisation; all gradients to 1e-5: each is a
    sum of some hundred FP32 terms of 2^-24 relative error, with decays of up
    to 300 steps' memory."""
    from fft_block_toeplitz_amd import layers

    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    p, h0, w, b = leaf(gen, 3, 290, 96), leaf(gen, 3, 48), leaf(gen, 48), leaf(gen, 48)
    mix = torch.randn(3, 290, 48, generator=gen, device="cuda")
    h, last = layers.recurrence(p[..., :48], p[..., 48:] + 2.0, h0)
    y = layers.group_norm(h, 6, w, b, activation="gelu")
    ((y * mix).sum() + last.sum()).backward()

    pd, hd, wd, bd = (t.detach().double().requires_grad_() for t in (p, h0, w, b))
    a = torch.sigmoid(pd[..., 48:] + 2.0)
    state, states = hd, []
    for t in range(290):
        state = a[:, t] * state + (1.0 - a[:, t]) * pd[:, t, :48]
        states.append(state)
    hr = torch.stack(states, 1)
    g = hr.reshape(3, 290, 6, 8)
    var, mean = torch.var_mean(g, (1, 3), correction=0, keepdim=True)
    z = ((g - mean) / torch.sqrt(var + 1e-5)).reshape(3, 290, 48) * wd + bd
    yr = torch.nn.functional.gelu(z)
    ((yr * mix).sum() + state.sum()).backward()
    assert off(y, yr.detach()) < 1e-5 and off(last, state.detach()) < 1e-5
    for mine, ref in ((p, pd), (h0, hd), (w, wd), (b, bd)):
        assert off(mine.grad, ref.grad) < 1e-5


def test_gradients_that_are_absent_or_expanded(fm):
    """Only the last state is used; a gradient expanded from one number."""
    from fft_block_toeplitz_amd import layers

    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    x, g = leaf(gen, 2, 40, 16), leaf(gen, 2, 40, 16)
    h, last = layers.recurrence(x, g)
    last.sum().backward()
    only_last = x.grad.clone()
    x.grad = None
    layers.recurrence(x, g)[0][:, -1].sum().backward()
    assert torch.allclose(x.grad, only_last, rtol=1e-5, atol=1e-7)
    x.grad = None
    layers.group_norm(x, 4).sum().backward()  # the sum of a normalised group does not depend on x
    assert float(x.grad.abs().max()) < 1e-4


def test_layer_streams_what_it_computes_over_series(fm):
    from fft_block_toeplitz_amd.layers import RecurrentLayer

    torch.manual_seed(3)
    layer = RecurrentLayer(5, 40, 3, groups=4)
    x = torch.randn(3, 150, 5, device="cuda")
    with torch.no_grad():
        y, last = layer(x)
        front, middle = layer(x[:, :70])
        back, end = layer(x[:, 70:], middle)
    state = torch.zeros(3, 40, device="cuda")
    steps = torch.stack([layer.step(x[:, t], state) for t in range(150)], 1)
    for got, want in ((torch.cat([front, back], 1), y), (end, last), (steps, y), (state, last)):
        assert off(got, want.double()) < 1e-5
    short = torch.tensor([150, 20, 0], dtype=torch.int32, device="cuda")
    with torch.no_grad():
        _, ends = layer(x, lengths=short)
        _, want = layer(x[1:2, :20])
    assert off(ends[0], last[0].double()) < 1e-6 and off(ends[1], want[0].double()) < 1e-5
    assert not ends[2].any()


def test_surrogate_learns_the_operator_and_streams(fm):
    """The example end to end: the fit comes well under the zero model's error
    of 1, and the stream is the series to FP32 rounding."""
    from fft_block_toeplitz_amd import surrogate

    r = surrogate.run(iterations=150, Nt=120, report=None)
    assert r["fit"] < 0.3
    assert r["stream_against_series"] < 1e-5 and r["state_against_series"] < 1e-5


def test_layer_refuses_groups_that_do_not_divide(fm):
    from fft_block_toeplitz_amd.layers import RecurrentLayer

    with pytest.raises(ValueError):
        RecurrentLayer(4, 30, 2, groups=8)
