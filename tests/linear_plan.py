"""What the dense layers' C entry points launch, from a host build of
``csrc/linear.hip`` with its launches replaced by lines of text
(``cpp/linear_plan.cpp``): no GPU, nothing read at any address."""
import functools
import os
import shutil
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def hipcc():
    exe = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    return exe if os.path.exists(exe) else None


@functools.lru_cache(maxsize=None)
def _program():
    exe = os.path.join(tempfile.mkdtemp(prefix="linear_plan"), "linear_plan")
    subprocess.run([hipcc(), "--offload-arch=gfx950", "--offload-host-only", "-O1", "-std=c++17", f"-I{ROOT}/include",
                    f"-I{ROOT}/dense_gemm_optimisation_row_amd/csrc", "-x", "hip",
                    os.path.join(ROOT, "tests", "cpp", "linear_plan.cpp"), "-o", exe], check=True)
    return exe


def launches(calls):
    """For each call (a line of the program) its status, workspace and launches:
    (status, workspace, [{"kind": ..., fields}])."""
    out = subprocess.run([_program()], input="\n".join(calls) + "\n", capture_output=True, text=True, check=True).stdout
    found, now = [], []
    for line in out.splitlines():
        if line.startswith("status="):
            status, workspace = (int(f.split("=")[1]) for f in line.split())
            found.append((status, workspace, now))
            now = []
            continue
        kind, rest = line.split(" ", 1)
        rest = rest.replace("gated ", "gated_")
        now.append({"kind": kind, **{k: int(v) if v.lstrip("-").isdigit() else v
                                     for k, v in (f.split("=") for f in rest.split())}})
    assert len(found) == len(calls)
    return found


ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


def _ints(*v):
    return " ".join(str(int(i)) for i in v)


def linear(fmt, M, N, K, transposed=False, act="none", pad=0, x=0, w=0, y_f32=False):
    """The line of a call as ``dg.linear`` makes it; x, w: bytes of their bases
    past 16; pad: elements that every row has beyond its end."""
    ldw = (K if transposed else N) + pad
    return f"linear {fmt} {x} {w} 0 0 0 0 : " + _ints(M, N, K, transposed, K + pad, ldw, N + pad, N + pad, N + pad,
                                                     ACTS[act], y_f32)


def linear_backward(fmt, M, N, K, transposed=False, act="none", pad=0, dy=0, x=0, w=0, need=(True, True, True)):
    ld = (K if transposed else N)
    out = " ".join("0" if n else "-1" for n in need)
    return f"linear_backward {fmt} {dy} {x} {w} 0 {out} : " + _ints(M, N, K, transposed, N + pad, K + pad, ld + pad,
                                                                   N + pad, K, ld, ACTS[act])


def gated(fmt, M, F, K, transposed=False, act="silu", pad=0, x=0, w=0):
    ldw = (K if transposed else F) + pad
    return f"gated {fmt} {x} {w} {w} 0 0 0 : " + _ints(M, F, K, transposed, K + pad, ldw, F + pad, F, ACTS[act])


def gated_backward(fmt, M, F, K, transposed=False, act="silu", pad=0, x=0, w=0, need=(True, True), rounded=False):
    ld = (K if transposed else F)
    out = " ".join("0" if n else "-1" for n in (need[0], need[1], need[1]))
    return f"gated_backward {fmt} 0 {x} {w} {w} 0 0 {out} : " + _ints(M, F, K, transposed, F + pad, K + pad, ld + pad,
                                                                     F + pad, K, ld, ACTS[act] | (0x100 if rounded else 0))
