"""The differentiable forms on gradients, tensors and types that ordinary programs hand them."""
import pytest

from test_gpu_layers import leaf, off

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fft_block_toeplitz_amd as fm

    fm.lib()
    return fm


@pytest.mark.parametrize("how", ["sum over 1", "sum over 2", "transposed", "sum over 1 and 2", "channels"])
def test_norm_layer_takes_any_gradient_of_a_field(fm, how):
    """What sums and transposes behind a field of four dimensions hand back:
    gradients expanded over an axis, or with its axes in another order."""
    from fft_block_toeplitz_amd import layers

    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    x, w, b = leaf(gen, 2, 4, 5, 8), leaf(gen, 8), leaf(gen, 8)
    mix = torch.randn(2, 5, 4, 8, generator=gen, device="cuda")
    behind = {"sum over 1": lambda y, m: (y.sum(1) * m[:, :, 0]).sum(), "channels": lambda y, m: y.square().sum(3).sum(),
              "sum over 2": lambda y, m: (y.sum(2) * m[:, 0]).sum(), "transposed": lambda y, m: (y.transpose(1, 2) * m).sum(),
              "sum over 1 and 2": lambda y, m: (y.sum((1, 2)) * m[:, 0, 0]).sum()}[how]
    behind(layers.group_norm(x, 2, w, b, activation="silu"), mix).backward()
    xd, wd, bd = (t.detach().double().requires_grad_() for t in (x, w, b))
    v = xd.reshape(2, 20, 2, 4)
    var, mean = torch.var_mean(v, (1, 3), correction=0, keepdim=True)
    z = ((v - mean) / torch.sqrt(var + 1e-5)).reshape(2, 4, 5, 8) * wd + bd
    behind(z * torch.sigmoid(z), mix.double()).backward()
    for mine, ref in ((x, xd), (w, wd), (b, bd)):
        # sums of 40 FP32 terms, each some roundings of 6e-8
        assert off(mine.grad, ref.grad) < 1e-5


@pytest.mark.parametrize("shape", [(0, 3, 5, 8), (2, 0, 5, 8), (2, 3, 0, 8)])
def test_norm_of_empty_fields(fm, shape):
    from fft_block_toeplitz_amd import layers

    x, w = torch.zeros(shape, device="cuda").requires_grad_(), torch.ones(8, device="cuda").requires_grad_()
    y = layers.group_norm(x, 2, w, activation="gelu")
    y.sum().backward()
    assert y.shape == shape and x.grad.shape == shape and not w.grad.any()


def test_what_is_written_in_place_is_known_to_autograd(fm):
    """A state that a graph has saved, stepped on or written as `out` before
    the backward pass: an error, as for torch's own in-place operations, and
    not the gradient of other values."""
    from fft_block_toeplitz_amd import layers

    x = torch.randn(2, 30, 16, device="cuda", requires_grad=True)
    tokens = torch.randn(2, 16, device="cuda")

    def recurrence():
        state = torch.randn(2, 16, device="cuda")
        return layers.recurrence(x, x.detach() + 1.0, state)[0].sum(), state

    def product():
        kept = torch.randn(2, 30, 16, device="cuda")
        return (x * kept).sum(), kept

    for graph, write in (
            (recurrence, lambda t: fm.recurrence_step(tokens, tokens, t)),
            (recurrence, lambda t: fm.recurrence_step(tokens, tokens, t.clone(), out=t)),
            (product, lambda t: fm.recurrence(x.detach(), x.detach(), out=t)),
            (product, lambda t: fm.group_norm(x.detach(), 4, out=t))):
        loss, saved = graph()
        write(saved)
        with pytest.raises(RuntimeError, match="inplace|in-place"):
            loss.backward()
    # inference tensors have no versions; nothing to raise
    with torch.inference_mode():
        state = torch.zeros(2, 16, device="cuda")
        out = torch.empty(2, 16, device="cuda")
        assert fm.recurrence_step(tokens, tokens, state, out=out) is out and state.any()


def test_public_names_keep_gradients(fm):
    """fm.recurrence and fm.group_norm of tensors that require a gradient give
    results that have one; where there is none to give, they say so."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    x, g, h0, w, b = leaf(gen, 2, 40, 16), leaf(gen, 2, 40, 16), leaf(gen, 2, 16), leaf(gen, 16), leaf(gen, 16)
    leaves = (x, g, h0, w, b)

    def grads(m):
        h, last = m.recurrence(x, g, h0, decay="sigmoid", drive="plain")
        y = m.group_norm(h, 4, w, b, eps=1e-3, activation="gelu")
        return torch.autograd.grad(y.square().sum() + last.sum(), leaves)

    from fft_block_toeplitz_amd import layers

    for a, c in zip(grads(fm), grads(layers)):
        assert torch.equal(a, c)
    # one of the inputs is enough
    assert fm.recurrence(x.detach(), g.detach(), h0)[1].requires_grad
    assert fm.group_norm(x.detach(), 4, w).requires_grad and fm.group_norm(x.detach(), 4, bias=b).requires_grad
    # on another stream as well
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert fm.recurrence(x, g, stream=side)[0].requires_grad
    torch.cuda.current_stream().wait_stream(side)
    # without gradients nothing changes
    with torch.no_grad():
        assert not fm.recurrence(x, g)[0].requires_grad and not fm.group_norm(x, 4, w).requires_grad
        out = torch.empty_like(x)
        assert fm.recurrence(x, g, out=out)[0] is out
        fm.recurrence_step(x[:, 0], g[:, 0], torch.zeros(2, 16, device="cuda"))
    # save=True is the first half of a gradient by hand
    assert not any(t.requires_grad for t in fm.recurrence(x, g, save=True))
    assert not any(t.requires_grad for t in fm.group_norm(x, 4, w, save=True))
    state = torch.zeros(2, 16, device="cuda")
    for call in (lambda: fm.recurrence(x, g, out=torch.empty_like(x)), lambda: fm.group_norm(x, 4, out=torch.empty_like(x)),
                 lambda: fm.recurrence_step(x[:, 0], g[:, 0].detach(), state),
                 lambda: fm.recurrence_step(x[:, 0].detach(), g[:, 0].detach(), h0)):
        with pytest.raises(ValueError, match="gradient"):
            call()


@pytest.mark.parametrize("how", ["bfloat16", "half", "autocast"])
def test_layer_in_16_bits(fm, how):
    """The layer moved to a 16-bit type, or under autocast: trains and streams
    as in FP32, to that type's rounding."""
    from fft_block_toeplitz_amd.layers import RecurrentLayer

    torch.manual_seed(5)
    layer = RecurrentLayer(5, 40, 3, groups=4)
    x = torch.randn(3, 150, 5, device="cuda")
    want, want_last = layer(x)
    want.square().mean().backward()
    ref = [p.grad.clone() for p in layer.parameters()]
    layer.zero_grad()
    # a unit of bfloat16 is 2^-8; a few operations one after the other
    with torch.autocast("cuda", torch.bfloat16, enabled=how == "autocast"):
        if how != "autocast":
            layer, x = getattr(layer, how)(), getattr(x, how)()
        y, last = layer(x)
        y.square().mean().backward()
        state = torch.zeros(3, 40, device="cuda")
        steps = torch.stack([layer.step(x[:, t], state) for t in range(150)], 1)
    assert y.dtype == (torch.float16 if how == "half" else torch.bfloat16) and last.dtype == torch.float32
    assert off(y, want.detach().double()) < 16 * 2 ** -8 and off(steps, y.detach().double()) < 16 * 2 ** -8
    assert off(state, last.detach().double()) < 16 * 2 ** -8
    for p, r in zip(layer.parameters(), ref):
        assert p.grad.dtype == p.dtype and off(p.grad, r.double()) < 32 * 2 ** -8
