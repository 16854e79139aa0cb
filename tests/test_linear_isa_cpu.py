"""Checks on the generated gfx950 code of the dense layers' rings (CPU only):
as in the other rings, the loads that go straight to LDS are issued from
inline assembly that sets M0 and that the compiler's wait counters do not
see, so the compiler must keep nothing of its own in M0, spill nothing, and
hold the accumulators in their own registers."""
import os
import re
import shutil
import subprocess

import pytest

from dense_gemm_optimisation_row_amd import build as hipbuild


def _instances(src, name, tmp):
    if shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"):
        pytest.skip("hipcc not available")
    out = tmp.mktemp("isa") / (src + ".s")
    cmd = [hipbuild.hipcc(), *hipbuild.FLAGS, "-S", "--cuda-device-only", os.path.join(hipbuild.CSRC, src), "-o",
           str(out)]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    text = out.read_text()
    found = [(m.group(1), text[m.end():text.index(".Lfunc_end", m.end())])
             for m in re.finditer(rf"^(_Z\S*{name}\S*):.*$", text, flags=re.M)]
    assert found
    return text, found


@pytest.fixture(scope="module")
def ring(tmp_path_factory):
    return _instances("linear_ring.hip", "linear_ring_(?:pair_)?kernel", tmp_path_factory)


def test_every_layout_is_generated(ring):
    # two formats, five tiles; M x K with K x N and N x K, K x M with K x N,
    # gated with K x N and N x K; both products of a backward pass, three
    # tiles, with K x N and N x K
    assert sum("pair" not in sym for sym, _ in ring[1]) == 50
    assert sum("pair" in sym for sym, _ in ring[1]) == 12


def test_m0_is_touched_only_by_the_loads(ring):
    for sym, body in ring[1]:
        inside, loads = False, 0
        for line in body.splitlines():
            if "ASMSTART" in line or "ASMEND" in line:
                inside = "ASMSTART" in line
                continue
            code = line.split(";")[0]
            assert inside or not re.search(r"\bm0\b", code), f"{sym}: {code}"
            loads += inside and "buffer_load_dwordx4" in code and " lds" in code
        assert loads > 0, sym


def test_nothing_spills(ring):
    asm, found = ring
    for sym, body in found:
        def resource(name):
            return int(re.search(rf"^\s*\.set\s+{re.escape(sym)}\.{name},\s*(\d+)", asm, flags=re.M).group(1))
        assert resource("private_seg_size") == 0, sym
        assert "scratch_" not in body, sym
        bm, bn = (int(v) for v in re.search(r"ELi(\d+)ELi(\d+)E", sym).groups())
        assert resource("num_agpr") >= bm * bn // 256, sym   # the accumulators of 256 lanes
