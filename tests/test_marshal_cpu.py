"""The extension module on the CPU: C functions stand in for the entry points."""
import ctypes
import struct
import threading
import time

import pytest
import torch  # noqa: F401  (before the module, which is linked against it)

marshal = pytest.importorskip("dense_gemm_optimisation_row_amd._marshal")

LIBC = ctypes.CDLL(None)
NOTHING = (None, None, None)


def address(f):
    return ctypes.cast(f, ctypes.c_void_p).value


def kept(op, seconds):
    """A form whose entry point, nanosleep(parameters, NULL, ...), waits."""
    params = struct.pack("qq", int(seconds), int(seconds % 1 * 1e9))
    marshal.keep(op, NOTHING, (), 0, address(LIBC.nanosleep), params, (0, 1, 2), (), -1)


def test_other_threads_run_while_a_call_waits():
    kept(1000, 2.0)
    assert marshal.run(1001, NOTHING, (), 0, 0) is None      # of no such form
    done = threading.Event()
    t = threading.Thread(target=lambda: (marshal.run(1000, NOTHING, (), 0, 0), done.set()))
    start = time.perf_counter()
    t.start()
    while time.perf_counter() - start < 0.1:
        time.sleep(0.001)
    waiting = not done.is_set() and time.perf_counter() - start < 1.5
    t.join()
    assert waiting, "the interpreter stood still during the call"


def test_a_form_outlives_its_removal_during_a_call():
    kept(1002, 0.3)
    found = []
    t = threading.Thread(target=lambda: found.append(marshal.run(1002, NOTHING, (), 0, 0)))
    t.start()
    time.sleep(0.05)
    for op in range(2000, 2000 + 5000):       # more forms than are kept: all are dropped
        kept(op, 0)
    t.join()
    assert found == [()]
    assert marshal.run(1002, NOTHING, (), 0, 0) is None


def test_a_status_is_returned():
    marshal.keep(1003, NOTHING, (), 0, address(LIBC.nanosleep), struct.pack("qq", -1, 0), (0, 1, 2), (), -1)
    assert marshal.run(1003, NOTHING, (), 0, 0) == -1        # EINVAL
