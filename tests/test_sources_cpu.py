"""What a header of the kernels defines is not defined again by those that include it: a
copy would hide it, and a change to one would not reach the other."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_gemm_optimisation_row_amd", "csrc")
HEADERS = ("epilogue.h", "lds_dma.h", "ring.h")


def text(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def defined(source):
    """Names of structs and device functions at the outer level."""
    return set(re.findall(r"^struct (\w+)[^;]*\{", source, flags=re.M)) | \
        set(re.findall(r"^__device__ __forceinline__ [\w<> ]+?[ *&](\w+)\(", source, flags=re.M))


def included(name, seen=()):
    out = set()
    for h in re.findall(r'^#include "(\w+\.h)"', text(name), flags=re.M):
        if h not in seen and os.path.exists(os.path.join(CSRC, h)):
            out |= {h} | included(h, (*seen, h))
    return out


@pytest.mark.parametrize("name", sorted(n for n in os.listdir(CSRC) if n.endswith(".hip")))
def test_no_helper_of_a_header_is_defined_again(name):
    own, headers = defined(text(name)), included(name)
    for h in HEADERS:
        if h in headers:
            assert not own & defined(text(h)), (name, h)


def test_names_are_found():
    assert {"OpHalf", "OpBrain", "row_swizzle"} <= defined(text("ring.h"))
    assert {"Half16", "load8_of", "store8_of", "load8_f32", "activate"} <= defined(text("epilogue.h"))
    assert {"epilogue.h", "ring.h"} <= included("i8_kernels.hip") & included("orthogonalize.hip")
