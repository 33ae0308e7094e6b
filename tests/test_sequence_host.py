"""The torch layer of the sequence operators on the host: workspaces shared by
threads, and the checks that need no device. CPU only."""
import gc
import threading
import time
import weakref

import pytest

torch = pytest.importorskip("torch")

from fft_block_toeplitz_amd import sequence as sq  # noqa: E402


@pytest.fixture
def shared(monkeypatch):
    """The stream's workspace made on the CPU, slowly enough that threads meet in it."""
    monkeypatch.setattr(sq, "_workspaces", {})
    monkeypatch.setattr(sq._torch_module().cuda, "is_current_stream_capturing", lambda: False)
    zeros = torch.zeros

    def slow(*args, **kwargs):
        time.sleep(0.002)
        return zeros(*args, **kwargs)

    monkeypatch.setattr(torch, "zeros", slow)
    return torch.empty(0)


def test_threads_of_one_stream_share_a_workspace_safely(shared):
    """Calls of growing and changing sizes from eight threads: every call has
    a number of its own, in the order of the launches, and its counters and
    words are alive and as large as it asked for when it is launched, and still
    the stream's own: no other thread has replaced them."""
    launched, errors = [], []
    start = threading.Barrier(8)

    def launch(few, many, counters, counter_bytes, words, word_bytes, call):
        kept = {t.data_ptr(): t.numel() for t in gc.get_objects() if type(t) is torch.Tensor and t.dtype is torch.uint8}
        if kept.get(counters, 0) < few or kept.get(words, 0) < many or counter_bytes < few or word_bytes < many:
            errors.append("memory of a call that is about to be launched was freed")
        if not any(w[0] == counters and w[2] == words for w in sq._workspaces.values()):
            errors.append("a call uses a workspace that is not the stream's any more")
        launched.append((words, call))
        time.sleep(0.0005)

    def work(k):
        start.wait()
        for i in range(12):
            few, many = 256 * (1 + (k + i) % 3), 4096 * (1 + (3 * k + 5 * i) % 11)
            with sq._workspace((1, few, many), 0, 0, shared) as w:
                launch(few, many, *w)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[0]
    by_memory = {}
    for words, call in launched:
        by_memory.setdefault(words, []).append(call)
    for calls in by_memory.values():
        assert calls == sorted(set(calls)), "numbers repeat or run backwards"


def test_a_call_without_a_workspace_takes_none(shared):
    for _ in range(2):
        with sq._NO_WORKSPACE as (*memory, call):
            assert memory == [0, 0, 0, 0] and call == 0
    assert not sq._workspaces


def test_captured_calls_hold_memory_of_their_own(shared, monkeypatch):
    """Two captured calls: not the stream's workspace, alive until launched."""
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    made = []
    zeros = torch.zeros

    def watched(*args, **kwargs):
        t = zeros(*args, **kwargs)
        made.append(weakref.ref(t))
        return t

    monkeypatch.setattr(torch, "zeros", watched)
    for _ in range(2):
        with sq._workspace((1, 256, 512), 0, 0, shared) as w:
            assert [r().data_ptr() for r in made] == [w[0], w[2]] and w[4] == 1
        made.clear()
    assert not sq._workspaces


def test_numbers_start_again_on_a_cleared_workspace(shared):
    with sq._workspace((1, 256, 512), 0, 0, shared) as w:
        assert w[4] == 1
    entry = next(iter(sq._workspaces.values()))
    entry[4] = 2 ** 32 - 1
    entry[6].fill_(255)
    with sq._workspace((1, 256, 512), 0, 0, shared) as w:
        assert w[4] == 1 and not entry[6].any()


def test_overlap_of_an_output(monkeypatch):
    """Bytes shared with any input: contiguous, strided or a view of another type; neighbours are none."""
    flat = torch.zeros(100)
    out, like = flat[20:60].view(4, 10), torch.zeros(4, 10)
    assert sq._output(out, like, (flat[:20], None, flat[60:], flat.view(torch.int32)[60:70])) is out
    strided = flat[:60].view(6, 10)[:3, :5]  # its last element is flat[24]
    for other in (out, flat[59:], flat[:21], strided, flat[15:].as_strided((2,), (10,)), flat.view(torch.int32)[30:31]):
        with pytest.raises(ValueError, match="overlap"):
            sq._output(out, like, (like, None, other))
    assert sq._output(out, like, (flat[:50].view(5, 10)[:2, :5], flat[40:40])) is out  # ends at flat[14]; nothing at all


def test_rows_of_fields():
    """[samples, rows, channels] of every number of axes, empty ones too; rows that are not evenly spaced are refused."""
    for shape in ((3, 8), (3, 4, 8), (3, 4, 5, 8), (2, 3, 4, 5, 8), (0, 4, 5, 8), (3, 0, 5, 8), (3, 4, 0, 8), (3, 4, 5, 0)):
        v = sq._samples(torch.zeros(shape))
        assert v.shape == (shape[0], torch.Size(shape[1:-1]).numel(), shape[-1])
    x = torch.zeros(2, 4, 5, 8)
    assert sq._samples(x[:, :, :, :3]).stride() == (160, 8, 1)
    for uneven in (x.transpose(1, 2), x[:, :, :3], x.sum(1, keepdim=True).expand(2, 4, 5, 8)):
        with pytest.raises(ValueError, match="evenly"):
            sq._samples(uneven)
