"""The C entry points of the gated delta rule and of the queries' and keys'
norms refuse bad arguments before any device work, and their kernels spill no
vector registers. CPU only: no call here reaches a kernel."""
import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

import fft_block_toeplitz_amd as fm
from fft_block_toeplitz_amd import build as fbuild
from fft_block_toeplitz_amd import delta as dl
from fft_block_toeplitz_amd import sequence as sq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # never dereferenced
BIG = 2 ** 31


@pytest.fixture(scope="module")
def lib():
    if fbuild.is_stale():
        fbuild.build()
    return dl._lib()


def heads(name):
    return f"{name} {name}_batch {name}_step {name}_head"


def field(name, step, head):
    return {name: FAKE, name + "_batch": 100 * step, name + "_step": step, name + "_head": head}


DELTA = "batch steps key_heads heads keys values dtype decay rate scale lengths offsets " + " ".join(
    heads(f) for f in "q k v gate beta".split()) + " h0 carries workspace workspace_bytes " + heads("y") + " h_last " + \
    heads("dy") + " dh_last " + " ".join(heads(f) for f in "dq dk dv dgate dbeta".split()) + " dh0"
STEP = "batch key_heads heads keys values places dtype decay rate scale " + " ".join(
    heads(f) for f in "q k v gate beta".split()) + " state state_place slots " + heads("y")
NORM = "batch steps query_heads key_heads dim frequencies dtype norm pairs eps lengths frequency positions position_batch " \
    + heads("q") + " " + heads("k") + " q_weight k_weight " + " ".join(
        heads(f) for f in "qy ky dqy dky dq dk".split()) + " dq_weight dk_weight workspace workspace_bytes"
KEYED, VALUED, GATES = dict(step=32, head=16), dict(step=32, head=8), dict(step=4, head=1)
INPUTS = {**field("q", **KEYED), **field("k", **KEYED), **field("v", **VALUED), **field("gate", **GATES),
          **field("beta", **GATES)}
FIELDS = {
    "delta": (dl._DELTA, DELTA, dict(
        batch=2, steps=100, key_heads=2, heads=4, keys=16, values=8, scale=1.0, carries=FAKE, workspace=FAKE,
        workspace_bytes=1 << 40, **INPUTS, **field("y", **VALUED), **field("dy", **VALUED), **field("dq", **KEYED),
        **field("dk", **KEYED), **field("dv", **VALUED), **field("dgate", **GATES), **field("dbeta", **GATES))),
    "step": (dl._DELTA_STEP, STEP, dict(batch=2, key_heads=2, heads=4, keys=16, values=8, places=3, scale=1.0, **INPUTS,
                                        state=FAKE, state_place=512, **field("y", **VALUED))),
    "norm": (dl._QK_NORM, NORM, dict(
        batch=2, steps=10, query_heads=2, key_heads=2, dim=16, frequencies=8, eps=1e-6, frequency=FAKE, positions=FAKE,
        position_batch=10, workspace=FAKE, workspace_bytes=1 << 30, dq_weight=FAKE, dk_weight=FAKE,
        **{k: v for f in "q k qy ky dqy dky dq dk".split() for k, v in field(f, **KEYED).items()})),
}


def packed(kind, **change):
    layout, names, good = FIELDS[kind]
    values = {**dict.fromkeys(names.split(), 0), **good, **change}
    return layout.pack(*(values[n] for n in names.split()))


def test_structures_match_the_header(tmp_path):
    """Sizes and late offsets, as the C compiler lays the structures out."""
    if not shutil.which("gcc"):
        pytest.skip("gcc not available")
    src = tmp_path / "sizes.c"
    asked = [("delta", "delta_rule", "h_last"), ("delta", "delta_rule", "dh_last"), ("delta", "delta_rule", "dh0"),
             ("step", "delta_rule_step", "slots"), ("norm", "qk_norm", "q_weight"), ("norm", "qk_norm", "workspace_bytes")]
    types = ["fftmv_delta_rule_t", "fftmv_delta_rule_step_t", "fftmv_qk_norm_t"]
    values = [f"sizeof({t})" for t in types] + [f"offsetof(fftmv_{t}_t, {m})" for _, t, m in asked]
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#define __HIP_PLATFORM_AMD__\n#include "fftmv.h"\n'
                   "int main(void) { size_t v[] = {" + ", ".join(values) + "}; "
                   'for (size_t i = 0; i < sizeof v / sizeof *v; ++i) printf("%zu ", v[i]); return 0; }\n')
    exe = str(tmp_path / "sizes")
    subprocess.run(["gcc", f"-I{ROOT}/include", "-I/opt/rocm/include", str(src), "-o", exe], check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    mark = 0x7172737475767778
    assert got == [FIELDS[k][0].size for k in ("delta", "step", "norm")] + [
        packed(kind, **{m: mark}).index(mark.to_bytes(8, "little")) for kind, _, m in asked]


INVALID, UNSUPPORTED = fm.FFTMV_ERR_INVALID_ARG, fm.FFTMV_ERR_UNSUPPORTED_SIZE
COMMON = (dict(batch=0), dict(steps=-1), dict(key_heads=0), dict(key_heads=3), dict(heads=0), dict(keys=0), dict(values=0),
          dict(dtype=3), dict(dtype=-1), dict(decay=2), dict(rate=2), dict(lengths=FAKE, offsets=FAKE), dict(q=0),
          dict(k=FAKE + 1), dict(v=FAKE + 2), dict(gate=0), dict(beta=0), dict(q_step=-1), dict(k_head=-1),
          dict(v_batch=2 ** 62), dict(q_head=2 ** 62), dict(h0=FAKE + 2), dict(lengths=FAKE + 2), dict(offsets=FAKE + 1),
          dict(workspace=0), dict(workspace=FAKE + 8), dict(workspace_bytes=100))


@pytest.mark.parametrize("kind,entry,change,status", [
    *[("delta", e, c, INVALID) for e in ("rule_forward", "rule_backward") for c in COMMON],
    ("delta", "rule_forward", dict(y=0), INVALID), ("delta", "rule_forward", dict(h_last=FAKE + 1), INVALID),
    *[("delta", "rule_backward", c, INVALID) for c in (
        dict(dy=0), dict(dq=0), dict(dk=FAKE + 2), dict(dv=0), dict(dgate=0), dict(dbeta=0), dict(carries=0),
        dict(dh_last=FAKE + 2), dict(dh0=FAKE + 3))],
    *[("delta", "rule_forward", c, UNSUPPORTED) for c in (
        dict(keys=129), dict(values=1025), dict(batch=BIG), dict(steps=BIG), dict(heads=BIG, key_heads=1),
        dict(batch=2 ** 26, heads=64, key_heads=1), dict(steps=2 ** 30, batch=64),
        dict(steps=BIG, offsets=FAKE))],
    *[("step", "rule_step", c, INVALID) for c in (
        dict(batch=0), dict(places=0), dict(places=1), dict(heads=3), dict(dtype=5), dict(decay=-1), dict(rate=3),
        dict(q=0), dict(k=0), dict(v=FAKE + 1), dict(gate=0), dict(beta=0), dict(y=0), dict(state=0),
        dict(state=FAKE + 2), dict(state_place=511), dict(slots=FAKE + 2), dict(v_step=-1))],
    *[("step", "rule_step", c, UNSUPPORTED) for c in (dict(keys=200), dict(values=2000), dict(places=BIG))],
    *[("norm", e, c, INVALID) for e in ("norm_forward", "norm_backward") for c in (
        dict(batch=0), dict(steps=-1), dict(query_heads=0), dict(key_heads=-1), dict(dim=0), dict(frequencies=9),
        dict(frequencies=-1), dict(dtype=3), dict(norm=2), dict(pairs=2), dict(eps=-1.0), dict(eps=float("nan")),
        dict(q=0), dict(k=FAKE + 2), dict(q_step=-1), dict(frequency=0), dict(frequency=FAKE + 4),
        dict(positions=FAKE + 2), dict(position_batch=-1), dict(lengths=FAKE + 1), dict(q_weight=FAKE + 2),
        dict(dk_weight=FAKE + 1))],
    ("norm", "norm_forward", dict(qy=0), INVALID), ("norm", "norm_forward", dict(ky=0), INVALID),
    *[("norm", "norm_backward", c, INVALID) for c in (dict(dqy=0), dict(dky=0), dict(dq=0), dict(dk=0), dict(workspace=0),
                                                      dict(workspace_bytes=8))],
    *[("norm", "norm_forward", c, UNSUPPORTED) for c in (dict(dim=513, frequencies=0), dict(steps=BIG),
                                                         dict(batch=2 ** 16, steps=2 ** 16))],
])
def test_refusals_before_device_work(lib, kind, entry, change, status):
    name = {"norm": "fftmv_qk_"}.get(kind, "fftmv_delta_") + entry
    assert getattr(lib, name)(packed(kind, **change), None) == status


def test_null_structures_are_refused(lib):
    for name in ("delta_rule_forward", "delta_rule_backward", "delta_rule_step", "qk_norm_forward", "qk_norm_backward"):
        assert getattr(lib, "fftmv_" + name)(None, None) == INVALID


def test_sizes(lib):
    assert dl.fftmv_delta_rule_sizes(3, 0, 1, 1, 8, 8, 0, False, False) == (0, 0)
    assert dl.fftmv_delta_rule_sizes(3, 0, 1, 1, 8, 8, 0, True, True) == (0, 0)
    assert dl.fftmv_delta_rule_sizes(3, 65, 1, 2, 8, 8, 1, False, False)[0] == 6
    assert dl.fftmv_delta_rule_sizes(3, 65, 1, 2, 8, 8, 1, True, False)[0] == 4
    forward, backward = (dl.fftmv_delta_rule_sizes(2, 500, 2, 4, 64, 32, 0, False, b)[1] for b in (False, True))
    assert backward >= forward + 16 * 4 * 64 * 32 * 4 > 0
    with pytest.raises(fm.FftmvError):
        dl.fftmv_delta_rule_sizes(1, 1, 2, 3, 8, 8, 0, False, False)
    assert lib.fftmv_delta_rule_sizes(1, 300, 1, 1, 8, 8, 0, 0, 0, None, None) == fm.FFTMV_SUCCESS
    assert dl.fftmv_qk_norm_workspace(2, 3, 1, 1, 10) >= 2 * 6 * 10 * 4
    assert lib.fftmv_qk_norm_workspace(1, 1, 1, 1, 8, None) == INVALID


def test_no_kernel_spills_vector_registers(tmp_path):
    if not os.path.exists(fbuild.HIPCC):
        pytest.skip("hipcc not available")
    sources = [s for s in fbuild.SOURCES if re.search(r"/(delta_rule|qk_norm)\w*\.hip$", s)]
    assert len(sources) == 8

    def report(src):
        cmd = [fbuild.HIPCC, *fbuild.FLAGS, f"-I{os.path.join(ROOT, 'include')}", "--cuda-device-only",
               "-Rpass-analysis=kernel-resource-usage", "-c", src, "-o", str(tmp_path / (os.path.basename(src) + ".o"))]
        res = subprocess.run(cmd, capture_output=True, text=True)
        assert res.returncode == 0, res.stderr[-2000:]
        return [(src, int(n)) for n in re.findall(r"VGPRs Spill: (\d+)", res.stderr)]

    with ThreadPoolExecutor(max(1, min(8, int(os.environ.get("MAX_JOBS", os.cpu_count() or 1))))) as ex:
        found = [v for r in ex.map(report, sources) for v in r]
    assert len(found) > 50
    assert not [v for v in found if v[1]], "kernels with spilled registers"


def test_numbers_of_the_header(lib):
    text = open(os.path.join(ROOT, "include", "fftmv.h")).read()
    defined = dict(re.findall(r"#define (FFTMV_\w+) (\d+)", text))
    for name in ("FFTMV_DELTA_RUN", "FFTMV_DELTA_KEYS", "FFTMV_DELTA_VALUES", "FFTMV_QK_NORM_DIM"):
        assert int(defined[name]) == getattr(dl, name)
    for table, prefix in ((dl.RATES, "RATE"), (dl.NORMS, "NORM"), (dl.PAIRS, "PAIRS"), (dl.DECAYS, "DECAY")):
        for name, value in table.items():
            assert int(defined[f"FFTMV_{prefix}_{name.upper()}"]) == value
    assert sq.DECAYS["sigmoid"] == dl.DECAYS["sigmoid"] and sq.DECAYS["exp"] == dl.DECAYS["exp"]
