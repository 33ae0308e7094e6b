"""The tolerance of the gates' gradients (delta_exact) takes the definition's result rounded once and nothing that is
merely near it: not zeros, not the opposite, not a tenth or a hundredth more, not the neighbouring step's. CPU only."""
import pytest

torch = pytest.importorskip("torch")

import delta_exact as E  # noqa: E402


def inputs(seed, T, Hk, H, K, V, dtype, spread=None):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    q, k = (torch.nn.functional.normalize(n(T, Hk, K), dim=-1) for _ in range(2))
    gate = n(T, H) + 2.0 + 3.0 * torch.rand(H, generator=gen) if spread is None else spread * n(T, H)
    x = [t.to(dtype).double() for t in (q, k, n(T, H, V), gate, n(T, H))]
    return x, n(H, K, V).double(), n(T, H, V).to(dtype).double(), n(H, K, V).double()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,Hk,H,K,V,spread", [(150, 2, 2, 64, 64, None), (70, 1, 1, 16, 1024, None), (64, 1, 1, 128, 128, None),
                                               (200, 1, 1, 128, 200, None), (150, 1, 2, 64, 64, 4.0), (3, 1, 1, 25, 25, None)])
def test_what_the_tolerance_rejects(dtype, T, Hk, H, K, V, spread):
    x, h0, dy, dlast = inputs(T, T, Hk, H, K, V, dtype, spread)
    r = E.gradients(*x, h0, "sigmoid", "sigmoid", K ** -0.5, dy, dlast)
    for h in range(H):
        want, size = r["dgate"][:, h], r["size"][:, h]
        assert E.gates_off(want.to(dtype), want, size, dtype) is None
        for wrong in (torch.zeros_like(want), -want, 1.1 * want, 1.016 * want, want.roll(1), want * float("nan")):
            assert E.gates_off(wrong.to(dtype), want, size, dtype) is not None


def test_gradients_of_the_reference():
    """The reference's gradients against automatic differentiation."""
    x, h0, dy, dlast = inputs(3, 70, 2, 4, 6, 5, torch.float32)
    r = E.gradients(*x, h0, "sigmoid", "sigmoid", 0.3, dy, dlast)
    leaves = [t.requires_grad_() for t in (*x, h0)]
    q, k, v, gate, beta, state = leaves
    y = []
    for t in range(70):
        kt, qt = (z[t].repeat_interleave(2, 0) for z in (k, q))
        pre = torch.sigmoid(gate[t])[:, None, None] * state
        state = pre + torch.sigmoid(beta[t])[:, None, None] * kt[:, :, None] * (v[t] - (pre * kt[:, :, None]).sum(1))[:, None]
        y.append(0.3 * (state * qt[:, :, None]).sum(1))
    y = torch.stack(y)
    torch.testing.assert_close(r["y"], y.detach(), rtol=1e-12, atol=1e-12)
    grads = torch.autograd.grad((y, state), leaves, (dy, dlast))
    for name, g in zip(("dq", "dk", "dv", "dgate", "dbeta", "dh0"), grads):
        torch.testing.assert_close(r[name], g, rtol=1e-10, atol=1e-12)
