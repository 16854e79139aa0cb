"""Checks on the generated gfx950 code of the 8-bit rings and of the orthogonalised
update's products (CPU only), as for the dense layers' rings: nothing of the
compiler's in M0, no spills, the accumulators in their own registers."""
import re

import pytest

from test_linear_isa_cpu import _instances

KERNELS = {"i8_ring_kernel": ("i8_kernels.hip", 8, True), "i8_rows_kernel": ("i8_kernels.hip", 8, False),
           "newton_schulz_kernel": ("orthogonalize.hip", 12, True),
           "newton_schulz_small_kernel": ("orthogonalize.hip", 1, False),
           "strips_start_kernel": ("orthogonalize.hip", 4, False), "strips_step_kernel": ("orthogonalize.hip", 8, False),
           "quantize_kernel": ("quantize.hip", 36, False)}


@pytest.fixture(scope="module", params=KERNELS)
def kernel(request, tmp_path_factory):
    src, count, direct = KERNELS[request.param]
    return (*_instances(src, request.param, tmp_path_factory), count, direct)


def test_every_variant_is_generated(kernel):
    # four tiles, one matrix and two; one to four blocks of rows, one matrix and two;
    # three products on three tiles, and on the smallest with and without sums apart;
    # a step of strips and the last, of one to four blocks of 32 rows
    assert len(kernel[1]) == kernel[2]


def test_m0_is_touched_only_by_the_loads(kernel):
    if not kernel[3]:
        pytest.skip("no loads straight to LDS")
    for sym, body in kernel[1]:
        inside, loads = False, 0
        for line in body.splitlines():
            if "ASMSTART" in line or "ASMEND" in line:
                inside = "ASMSTART" in line
                continue
            code = line.split(";")[0]
            assert inside or not re.search(r"\bm0\b", code), f"{sym}: {code}"
            loads += inside and "buffer_load_dwordx4" in code and " lds" in code
        assert loads > 0, sym


def test_nothing_spills(kernel):
    asm, found = kernel[:2]
    for sym, body in found:
        size = int(re.search(rf"^\s*\.set\s+{re.escape(sym)}\.private_seg_size,\s*(\d+)", asm, flags=re.M).group(1))
        assert size == 0 and "scratch_" not in body, sym
