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
