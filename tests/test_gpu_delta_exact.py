"""How exact the gated delta rule is: results of 16 bits are the definition's rounded once, and the gates' gradients are
as near as sums in 32 bits come (delta_exact), for each head by itself."""
import pytest

torch = pytest.importorskip("torch")

import delta_exact as E  # noqa: E402
from test_gpu_delta import DT, fields, generator  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fft_block_toeplitz_amd as fm

    fm.lib()
    return fm


def call(fm, seed, B, T, Hk, H, K, V, dtype, decay="sigmoid", rate="sigmoid", change=None, strided=False):
    """Results of one forward and backward call and, for each sequence, those of the definition."""
    x = fields(seed, (B, T), Hk, H, K, V, dtype, decay, rate, strided)
    gen = generator(seed + 500)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    h0, dlast, dy = n(B, H, K, V), n(B, H, K, V), n(B, T, H, V)
    if change:
        change(*x, dy, dlast)
    dy = dy.to(DT[dtype])
    y, last, carries = fm.delta_rule(*x, h0, decay=decay, rate=rate, save=True)
    grads = fm.delta_rule_backward(dy, *x, carries, h0, dlast, decay=decay, rate=rate)
    got = dict(zip(("y", "last", "dq", "dk", "dv", "dgate", "dbeta", "dh0"), (y, last, *grads)))
    want = [E.gradients(*(t[b].double() for t in x), h0[b].double(), decay, rate, K ** -0.5, dy[b].double(),
                        dlast[b].double()) for b in range(B)]
    return got, want


# A result in 32 bits is off by about 20 U of its head's mean, 0.8 times that without its sign (delta_exact), and rounds
# to another neighbour where a border lies between: with steps of 2^-7.5 of a value on average for bf16, and the mean
# over 1 / |value| of normal values, of which one in ten thousand is the smallest, 7.3:
#   0.8 * 20 * 2^-24 * 2^7.5 * 7.3 = 1.3e-3, and eight times as much for fp16, whose steps are an eighth
FLIPS = {"bf16": 1.3e-3, "fp16": 1.04e-2}


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B,T,Hk,H,K,V,strided", [
    (1, 300, 4, 4, 128, 128, False), (2, 200, 1, 4, 128, 64, False), (2, 300, 2, 4, 64, 64, False),
    (3, 250, 2, 2, 32, 80, False), (1, 250, 3, 3, 75, 41, True), (1, 250, 1, 3, 100, 72, True),
    (1, 640, 1, 1, 128, 128, False), (1, 250, 1, 2, 33, 200, False)])
def test_results_round_once(fm, dtype, B, T, Hk, H, K, V, strided):
    got, want = call(fm, 31, B, T, Hk, H, K, V, dtype, strided=strided)
    for name in ("y", "dq", "dk", "dv"):
        ref = torch.stack([w[name] for w in want]).to(DT[dtype])
        flips = float((got[name] != ref).double().mean())
        assert flips <= FLIPS[dtype], f"{name}: {flips:.2g} of the values round to another neighbour"


SHAPES = [(1, 1, 1, 1, 1, 1), (2, 3, 1, 1, 25, 25), (2, 150, 2, 2, 64, 64), (1, 200, 2, 6, 64, 64), (1, 70, 1, 1, 16, 1024),
          (1, 64, 1, 1, 128, 128), (1, 130, 1, 4, 128, 128), (1, 300, 1, 1, 128, 200), (1, 200, 3, 3, 75, 41),
          (1, 640, 1, 2, 32, 33), (1, 130, 1, 3, 100, 40)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("B,T,Hk,H,K,V", SHAPES)
def test_gradients_of_gates(fm, dtype, B, T, Hk, H, K, V):
    for decay in ("sigmoid", "exp"):
        got, want = call(fm, 32 + T, B, T, Hk, H, K, V, dtype, decay)
        for b in range(B):
            for h in range(H):
                wrong = E.gates_off(got["dgate"][b, :, h], want[b]["dgate"][:, h], want[b]["size"][:, h], DT[dtype])
                assert not wrong, f"{decay}, sequence {b}, head {h}: {wrong}"


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("Hk,H,K,V", [(2, 2, 64, 64), (1, 2, 64, 64), (2, 2, 128, 128), (1, 3, 128, 64), (2, 4, 24, 40)])
def test_gradients_of_gates_far_apart(fm, dtype, Hk, H, K, V):
    """Gates between one that forgets in a step and one that keeps hundreds: small gradients beside large ones."""
    def change(q, k, v, gate, beta, dy, dlast):
        gate.copy_(4.0 * torch.randn(gate.shape, generator=generator(5), device="cuda"))

    got, want = call(fm, 33, 2, 200, Hk, H, K, V, dtype, change=change)
    for b in range(2):
        for h in range(H):
            wrong = E.gates_off(got["dgate"][b, :, h], want[b]["dgate"][:, h], want[b]["size"][:, h], DT[dtype])
            assert not wrong, f"sequence {b}, head {h}: {wrong}"


@pytest.mark.parametrize("dtype,small", [("bf16", -20), ("fp16", -10), ("fp32", -20)])
@pytest.mark.parametrize("K,V", [(24, 40), (64, 64), (128, 72)])
def test_gradients_of_gates_beside_a_larger_head(fm, dtype, small, K, V):
    """A head whose outputs count far less than those of the head in front of it, with the same queries and keys: the
    larger one's roundings stay out of its gates' gradients, in either order."""
    for first in (True, False):
        def change(q, k, v, gate, beta, dy, dlast):
            one, rest = (slice(0, 1), slice(1, 3)) if first else (slice(2, 3), slice(0, 2))
            for t, heads in ((dy, 2), (dlast, 1)):
                t.movedim(heads, 0)[rest] *= 2.0 ** small
                t.movedim(heads, 0)[one] *= 8.0

        got, want = call(fm, 34, 1, 150, 1, 3, K, V, dtype, change=change)
        for h in range(3):
            wrong = E.gates_off(got["dgate"][0, :, h], want[0]["dgate"][:, h], want[0]["size"][:, h], DT[dtype])
            assert not wrong, f"head {h}: {wrong}"


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("K,V", [(32, 72), (64, 64), (128, 40)])
def test_not_finite_in_any_head_of_a_group(fm, bad, dtype, K, V):
    """One value that is not finite, in each head of a group in turn: the others' values, gates and rates keep their
    gradients' bits."""
    x = fields(35, (2, 200), 2, 6, K, V, dtype)
    dy = torch.randn((2, 200, 6, V), generator=generator(36), device="cuda").to(DT[dtype])
    y, last, carries = fm.delta_rule(*x, save=True)
    grads = fm.delta_rule_backward(dy, *x, carries)
    for head in (0, 1, 2, 4):
        for t in (x[2], dy):
            kept = t[1, 130, head, 5].clone()
            t[1, 130, head, 5] = bad
            y2, last2, carries2 = fm.delta_rule(*x, save=True)
            grads2 = fm.delta_rule_backward(dy, *x, carries2)
            t[1, 130, head, 5] = kept
            rest = [h for h in range(6) if h != head]
            assert not torch.isfinite(grads2[3][1, :, head]).all()
            for a, b in ((y2, y), *zip(grads2[2:5], grads[2:5])):
                assert torch.equal(a[0], b[0]) and torch.equal(a[1, :, rest], b[1, :, rest])
            for a, b in ((last2, last), (grads2[5], grads[5])):
                assert torch.equal(a[0], b[0]) and torch.equal(a[1, rest], b[1, rest])
            for a, b in zip(grads2[:2], grads[:2]):
                group = head // 3
                assert torch.equal(a[0], b[0]) and torch.equal(a[1, :, 1 - group], b[1, :, 1 - group])
