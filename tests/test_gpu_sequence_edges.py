"""The sequence operators at the edges of what their entry points accept."""
import numpy as np
import pytest

import sequence_reference as R

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
