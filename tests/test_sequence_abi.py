"""The sequence operators' C entry points refuse bad arguments before any
device work, and no kernel of theirs spills registers. CPU only: no call here
reaches a kernel."""
import ctypes
import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

import fft_block_toeplitz_amd as fm
from fft_block_toeplitz_amd import build as fbuild
from fft_block_toeplitz_amd import sequence as sq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    if fbuild.is_stale():
        fbuild.build()
    return sq._lib()


FIELDS = {
    "recurrence": (sq._RECURRENCE, "batch steps channels dtype decay drive call lengths offsets x x_batch x_step gate "
                   "gate_batch gate_step h0 carries counters counter_bytes workspace workspace_bytes h h_batch h_step "
                   "h_last dh dh_batch dh_step dh_last dx dx_batch dx_step dgate dgate_batch dgate_step dh0",
                   dict(batch=2, steps=300, channels=8, call=1, x=FAKE, x_batch=2400, x_step=8, gate=FAKE,
                        gate_batch=2400, gate_step=8, carries=FAKE, counters=FAKE, counter_bytes=1 << 20,
                        workspace=FAKE, workspace_bytes=1 << 30, h=FAKE, h_batch=2400, h_step=8, dh=FAKE,
                        dh_batch=2400, dh_step=8, dx=FAKE, dx_batch=2400, dx_step=8, dgate=FAKE, dgate_batch=2400,
                        dgate_step=8)),
    "step": (sq._STEP, "batch channels places dtype decay drive reserved x x_step gate gate_step state state_step "
             "slots h h_step",
             dict(batch=2, channels=8, places=4, x=FAKE, x_step=8, gate=FAKE, gate_step=8, state=FAKE, state_step=8,
                  h=FAKE, h_step=8)),
    "group_norm": (sq._GROUP_NORM, "samples rows channels groups dtype activation eps reserved lengths x x_sample "
                   "x_row weight bias stats workspace workspace_bytes y y_sample y_row dy dy_sample dy_row dx "
                   "dx_sample dx_row dweight dbias",
                   dict(samples=2, rows=5, channels=8, groups=2, eps=1e-5, x=FAKE, x_sample=40, x_row=8, stats=FAKE,
                        workspace=FAKE, workspace_bytes=1 << 30, y=FAKE, y_sample=40, y_row=8, dy=FAKE, dy_sample=40,
                        dy_row=8, dx=FAKE, dx_sample=40, dx_row=8, dweight=FAKE, dbias=FAKE)),
}


def packed(kind, **change):
    layout, names, good = FIELDS[kind]
    values = {**dict.fromkeys(names.split(), 0), **good, **change}
    return layout.pack(*(values[n] for n in names.split()))


def test_structures_match_the_header(tmp_path):
    """Sizes and last offsets, as the C compiler lays the structures out."""
    if not shutil.which("gcc"):
        pytest.skip("gcc not available")
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#define __HIP_PLATFORM_AMD__\n#include "fftmv.h"\n'
                   'int main(void) { printf("%zu %zu %zu %zu %zu %zu\\n", sizeof(fftmv_recurrence_t), '
                   "sizeof(fftmv_recurrence_step_t), sizeof(fftmv_group_norm_t), offsetof(fftmv_recurrence_t, h), "
                   "offsetof(fftmv_recurrence_step_t, slots), offsetof(fftmv_group_norm_t, dweight)); return 0; }\n")
    exe = str(tmp_path / "sizes")
    subprocess.run(["gcc", f"-I{ROOT}/include", "-I/opt/rocm/include", str(src), "-o", exe], check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    r, s, g = (FIELDS[k][0] for k in ("recurrence", "step", "group_norm"))

    def offset(kind, name):  # where packing one mark puts it
        mark = 0x7172737475767778
        return packed(kind, **{name: mark}).index(mark.to_bytes(8, "little"))

    assert got == [r.size, s.size, g.size, offset("recurrence", "h"), offset("step", "slots"),
                   offset("group_norm", "dweight")]


BIG = 2 ** 31


@pytest.mark.parametrize("kind,entry,change,status", [
    *[("recurrence", e, c, fm.FFTMV_ERR_INVALID_ARG) for e in ("forward", "backward") for c in (
        dict(batch=0), dict(steps=-1), dict(channels=0), dict(dtype=3), dict(decay=3), dict(drive=2), dict(dtype=-1),
        dict(lengths=FAKE, offsets=FAKE), dict(x=0), dict(gate=0), dict(x=FAKE + 1), dict(gate=FAKE + 2),
        dict(x_step=-8), dict(x_batch=2 ** 62), dict(h0=FAKE + 2), dict(lengths=FAKE + 1), dict(workspace=0),
        dict(workspace_bytes=64), dict(counters=0), dict(counter_bytes=4), dict(workspace=FAKE + 4), dict(call=0))],
    ("recurrence", "forward", dict(h=0), fm.FFTMV_ERR_INVALID_ARG),
    ("recurrence", "backward", dict(dh=0), fm.FFTMV_ERR_INVALID_ARG),
    ("recurrence", "backward", dict(dx=0), fm.FFTMV_ERR_INVALID_ARG),
    ("recurrence", "backward", dict(dgate=FAKE + 2), fm.FFTMV_ERR_INVALID_ARG),
    ("recurrence", "backward", dict(carries=0), fm.FFTMV_ERR_INVALID_ARG),
    *[("recurrence", "forward", c, fm.FFTMV_ERR_UNSUPPORTED_SIZE) for c in (
        dict(batch=BIG), dict(steps=BIG), dict(channels=BIG), dict(steps=BIG - 1))],
    *[("step", "step", c, fm.FFTMV_ERR_INVALID_ARG) for c in (
        dict(batch=0), dict(channels=0), dict(places=0), dict(places=1), dict(dtype=7), dict(reserved=1), dict(x=0),
        dict(state=0), dict(state=FAKE + 2), dict(h=0), dict(state_step=7), dict(x_step=-1), dict(slots=FAKE + 1))],
    ("step", "step", dict(places=BIG), fm.FFTMV_ERR_UNSUPPORTED_SIZE),
    *[("group_norm", e, c, fm.FFTMV_ERR_INVALID_ARG) for e in ("norm_forward", "norm_backward") for c in (
        dict(samples=0), dict(rows=-1), dict(groups=3), dict(groups=0), dict(dtype=4), dict(activation=3),
        dict(eps=-1.0), dict(eps=float("nan")), dict(reserved=2), dict(x=0), dict(x=FAKE + 2), dict(weight=FAKE + 1),
        dict(x_row=-1))],
    ("group_norm", "norm_forward", dict(y=0), fm.FFTMV_ERR_INVALID_ARG),
    ("group_norm", "norm_backward", dict(stats=0), fm.FFTMV_ERR_INVALID_ARG),
    ("group_norm", "norm_backward", dict(dy=0), fm.FFTMV_ERR_INVALID_ARG),
    ("group_norm", "norm_backward", dict(samples=4096, rows=1, workspace_bytes=8), fm.FFTMV_ERR_INVALID_ARG),
    ("group_norm", "norm_forward", dict(rows=BIG), fm.FFTMV_ERR_UNSUPPORTED_SIZE),
])
def test_refusals_before_device_work(lib, kind, entry, change, status):
    name = {"step": "fftmv_recurrence_step"}.get(entry) or (
        f"fftmv_group_{entry}" if kind == "group_norm" else f"fftmv_recurrence_{entry}")
    assert getattr(lib, name)(packed(kind, **change), None) == status


def test_null_structures_are_refused(lib):
    for name in ("recurrence_forward", "recurrence_backward", "recurrence_step", "group_norm_forward",
                 "group_norm_backward"):
        assert getattr(lib, "fftmv_" + name)(None, None) == fm.FFTMV_ERR_INVALID_ARG


def test_sizes(lib):
    assert sq.fftmv_recurrence_sizes(3, 0, 5, False) == (0, 0, 0)
    assert sq.fftmv_recurrence_sizes(7, 128, 5, False) == (0, 0, 0)  # no chunk follows another
    carries, counters, words = sq.fftmv_recurrence_sizes(7, 129, 5, False)
    assert carries == 14 and counters >= 7 * 128 and words >= 14 * 3 * 8 * 5
    assert sq.fftmv_recurrence_sizes(7, 1000, 5, True)[0] == 8
    with pytest.raises(fm.FftmvError):
        sq.fftmv_recurrence_sizes(0, 1, 1, False)
    with pytest.raises(fm.FftmvError):
        sq.fftmv_group_norm_workspace(1, 1, 5, 2, sq.FFTMV_F32, False)
    assert sq.fftmv_group_norm_workspace(4, 1, 512, 4, sq.FFTMV_BF16, False) == 0
    for call in (lib.fftmv_recurrence_sizes, ):
        assert call(1, 300, 8, 0, None, None, None) == fm.FFTMV_SUCCESS
    assert lib.fftmv_group_norm_workspace(1, 1, 8, 2, 0, 0, None) == fm.FFTMV_ERR_INVALID_ARG


def test_group_norm_workspaces_for_every_shape(lib):
    """The plan covers all shapes: widths around a vector's and a
    workgroup's, few and many groups, rows and samples."""
    for dtype in (sq.FFTMV_F32, sq.FFTMV_BF16):
        for D in (1, 2, 3, 7, 8, 25, 64, 125, 500, 2047, 4096, 4099, 8192, 9000):
            for G in (1, 2, 3, 33, 257, 2000):
                for N, S in ((1, 1), (1, 7), (3, 64), (300, 1), (20000, 1), (2, 5000), (1, 0)):
                    for backward in (False, True):
                        n = sq.fftmv_group_norm_workspace(N, S, D * G, G, dtype, backward)
                        assert 0 <= n <= 8 * (N + 2048 + 64) * (D * G + G), (dtype, D, G, N, S, backward)


def test_no_kernel_spills_registers(tmp_path):
    """Spilled kernels cost more than the occupancy they buy, and one computed
    wrong values; the compiler's own report has to say zero for each."""
    if not os.path.exists(fbuild.HIPCC):
        pytest.skip("hipcc not available")
    sources = [s for s in fbuild.SOURCES if re.search(r"/(recurrence|group_norm)_\w+\.hip$", s)]
    assert len(sources) == 13

    def report(src):
        cmd = [fbuild.HIPCC, *fbuild.FLAGS, f"-I{os.path.join(ROOT, 'include')}", "--cuda-device-only",
               "-Rpass-analysis=kernel-resource-usage", "-c", src, "-o", str(tmp_path / (os.path.basename(src) + ".o"))]
        res = subprocess.run(cmd, capture_output=True, text=True)
        assert res.returncode == 0, res.stderr[-2000:]
        return [(src, int(n)) for n in re.findall(r"VGPRs Spill: (\d+)", res.stderr)]

    with ThreadPoolExecutor(max(1, min(8, int(os.environ.get("MAX_JOBS", os.cpu_count() or 1))))) as ex:
        found = [v for r in ex.map(report, sources) for v in r]
    assert len(found) > 100
    assert not [v for v in found if v[1]], "kernels with spilled registers"
