"""Calls of the sequence operators' torch forms and layers that are refused, or answered, whatever the sizes: tangents of
forward-mode differentiation, layers moved between devices, positions of any distance, tiny rows."""
import pytest

torch = pytest.importorskip("torch")

from torch.autograd import forward_ad  # noqa: E402

from test_gpu_delta import fields  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fft_block_toeplitz_amd as fm

    fm.lib()
    return fm


def calls(fm):
    """(call, its arguments) of every entry point, small."""
    q, k, v, gate, beta = fields(1, (2, 10), 2, 4, 16, 8, "fp32")
    state, w = torch.zeros((2, 4, 16, 8), device="cuda"), torch.ones(16, device="cuda")
    y, _, carries = fm.delta_rule(q, k, v, gate, beta, state, save=True)
    x, g, h = v.flatten(2), v.flatten(2) + 1.0, torch.zeros((2, 32), device="cuda")
    hy, _, kept = fm.recurrence(x, g, h, save=True)
    z, stats = fm.group_norm(x, 4, save=True)
    one = torch.ones(32, device="cuda")
    return [
        (fm.delta_rule, dict(q=q, k=k, v=v, gate=gate, beta=beta, h0=state)),
        (lambda **a: fm.delta_rule(save=True, **a), dict(q=q, k=k, v=v, gate=gate, beta=beta, h0=state)),
        (fm.delta_rule_backward, dict(dy=y, q=q, k=k, v=v, gate=gate, beta=beta, carries=carries, h0=state, dh_last=state)),
        (fm.delta_rule_step, dict(q=q[:, 0], k=k[:, 0], v=v[:, 0], gate=gate[:, 0], beta=beta[:, 0], state=state.clone())),
        (fm.qk_norm, dict(q=q, k=k, q_weight=w, k_weight=w)),
        (fm.qk_norm_backward, dict(dqy=q, dky=k, q=q, k=k, q_weight=w, k_weight=w)),
        (fm.recurrence, dict(x=x, gate=g, h0=h)),
        (fm.recurrence_backward, dict(dh=hy, x=x, gate=g, carries=kept, h0=h, dh_last=h)),
        (fm.recurrence_step, dict(x=x[:, 0], gate=g[:, 0], state=h.clone())),
        (lambda **a: fm.group_norm(groups=4, **a), dict(x=x, weight=one, bias=one)),
        (lambda **a: fm.group_norm_backward(groups=4, **a), dict(dy=z, x=x, stats=stats, weight=one, bias=one)),
    ]


def test_tangents_are_refused(fm):
    """Each tensor of each call as a dual one, under no_grad too; without one, a level changes nothing."""
    for call, args in calls(fm):
        with forward_ad.dual_level():
            call(**args)
            for name, t in args.items():
                dual = forward_ad.make_dual(t, torch.ones_like(t))
                with pytest.raises(ValueError, match="forward-mode"):
                    call(**{**args, name: dual})
                with torch.no_grad(), pytest.raises(ValueError, match="forward-mode"):
                    call(**{**args, name: dual})


def test_layer_moved_to_the_gpu(fm):
    """Made on the CPU, moved, and moved to another type: what a layer made there gives."""
    from fft_block_toeplitz_amd.layers import DeltaLayer

    for dtype in (torch.float32, torch.bfloat16):
        here = DeltaLayer(10, 4, 16, 24, 6, key_heads=2, base=100.0).to(dtype)
        moved = DeltaLayer(10, 4, 16, 24, 6, key_heads=2, base=100.0, device="cpu").cuda().to(dtype)
        moved.load_state_dict(here.state_dict())
        x = torch.randn((3, 20, 10), device="cuda", dtype=dtype)
        at = torch.full((3,), 5, dtype=torch.int32, device="cuda")
        with torch.no_grad():
            (y, last), (y2, last2) = here(x), moved(x)
            assert torch.equal(last, last2) and torch.equal(y, y2)
            assert torch.equal(here.step(x[:, 0], last, None, at), moved.step(x[:, 0], last2, None, at))


def test_gradients_of_norms_that_are_missing(fm):
    q, k = fields(2, (2, 10), 2, 4, 16, 8, "bf16")[:2]
    for args in ((q, None, q, k), (None, k, q, k), (q, k, q, None), (None, None, q, None)):
        with pytest.raises(ValueError):
            fm.qk_norm_backward(*args)
    assert fm.qk_norm_backward(q, None, q)[1] is None


def test_positions_of_any_distance(fm):
    """One row of positions for all sequences, rows apart, a column's single steps: what a contiguous copy gives."""
    freq = 10.0 ** -torch.arange(4, dtype=torch.float64, device="cuda")
    pos = torch.randint(0, 1000, (40, 30), dtype=torch.int32, device="cuda")
    for rows, at in (((3, 10), pos[0, :10].expand(3, 10)), ((3, 10), pos[:3, 5:15]), ((3, 1), pos[:3, 7:8]),
                     ((1, 10), pos[4:5, :10]), ((10,), pos[4, :10]), ((3, 10), pos[::2][:3, :10])):
        q, k = fields(3, rows, 2, 2, 16, 8, "fp32")[:2]
        how, copy = {"frequencies": freq, "positions": at}, {"frequencies": freq, "positions": at.contiguous()}
        for a, b in zip(fm.qk_norm(q, k, **how), fm.qk_norm(q, k, **copy)):
            assert torch.equal(a, b)
        for a, b in zip(fm.qk_norm_backward(q, k, q, k, **how)[:2], fm.qk_norm_backward(q, k, q, k, **copy)[:2]):
            assert torch.equal(a, b)
    q = fields(3, (3, 10), 2, 2, 16, 8, "fp32")[0]
    for at in (pos[:10, :3].T, pos[:3, :20:2], pos[0, :1].expand(3, 10)):
        with pytest.raises(ValueError):
            fm.qk_norm(q, frequencies=freq, positions=at)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("norm", ["rms", "l2"])
def test_norms_of_tiny_rows(fm, dtype, norm):
    """Rows whose squares add up to a subnormal number, without an eps: as long as any others. The sum is a multiple of
    2^-149 and off by 64 halves of it at most, a relative 64 * 2^-150 / 2^-128 at the least sum of them, 2^-16."""
    x = fields(4, (3, 10), 2, 2, 64, 8, dtype)[0]
    x = (x.float() * 2.0 ** -63).to(x.dtype)  # rows of 2^-63, squares 2^-126 together and less
    x[1] *= 0.5
    x[2] = (x[2].float() * 0.6).to(x.dtype)
    y = fm.qk_norm(x, norm=norm, eps=0.0)[0].double()
    wide = x.double()
    want = wide / (wide.square().mean(-1, keepdim=True) if norm == "rms" else wide.square().sum(-1, keepdim=True)).sqrt()
    off = float(((y - want).norm(dim=-1) / want.norm(dim=-1)).nan_to_num(float("inf")).max())
    assert off <= 2.0 ** -16 + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -22)
