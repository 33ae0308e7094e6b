"""The sequence operators at the edges of what their entry points accept."""
import threading

import pytest

from test_gpu_sequence import check_norm, fields

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
