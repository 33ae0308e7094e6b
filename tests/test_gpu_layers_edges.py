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
