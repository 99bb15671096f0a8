"""The signals between the warps of the distillation gradient's pipeline, explored
state by state on the CPU for one CTA (grad_signals_shim.cu): whatever the order
of the warps' steps and of the copies' arrivals, no warp uses a slice before its
row's copy is there or once another row's is under way, no barrier is signalled
for a row before all have signalled it for the last, and every row is finished.
Where a wait is given up, which may be at any time, the rows from there on are
void; but the warps stay in step and end, no copy begins where another is
landing, and none is in flight at the end.

The slices and the copies' mbarriers are the library's (grad_signals.cuh,
compiled for the host).  A wait for an mbarrier follows the hardware's rule: it
returns when the phase in progress has another parity than the one asked for.
The exchange of a cluster only delays warps B, which the exploration does too."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    out = str(tmp_path_factory.mktemp("shim") / "libgrad_signals.so")
    cmd = [nvcc, "-std=c++17", "-O2", "-shared", "-Xcompiler", "-fPIC", "-gencode", "arch=compute_103a,code=sm_103a",
           f"-I{os.path.join(ROOT, 'verify_dspark_markov_gb300', 'csrc')}",
           os.path.join(ROOT, "tests", "grad_signals_shim.cu"), "-o", out]
    subprocess.run(cmd, check=True, capture_output=True)
    lib = ctypes.CDLL(out)
    lib.grad_explore.argtypes = [ctypes.c_int, ctypes.c_uint, *[ctypes.c_int] * 3, ctypes.c_char_p, ctypes.c_int]
    lib.grad_explore.restype = ctypes.c_longlong
    return lib


def explore(lib, rows, masked, barriers, give_up=False, hasty=False):
    """masked: the rows of weight 0, as bits.  (states, fault)"""
    fault = ctypes.create_string_buffer(200)
    return lib.grad_explore(rows, masked, barriers, int(give_up), int(hasty), fault, len(fault)), fault.value.decode()


@pytest.mark.parametrize("masked", [0, 0b10, 0b1111111, 0b0010111, 0b0101010, 0b1010101, 0b0001000, 0b1100110])
def test_every_order_of_seven_rows(library, masked):
    states, fault = explore(library, 7, masked, library.grad_barriers())
    assert states > 10_000, fault


@pytest.mark.parametrize("masked", [0, 0b0010, 0b0110])
def test_every_order_with_a_wait_given_up(library, masked):
    states, fault = explore(library, 4, masked, library.grad_barriers(), True)
    assert states > 10_000, fault


@pytest.mark.parametrize("masked", [0, 0b10, 0b0010111])
def test_one_barrier_to_a_slice_would_be_found(library, masked):
    """The exploration sees the fault of three mbarriers, one to a slice, whose
    phases two warps would wait for in turn."""
    states, fault = explore(library, 7, masked, 3)
    assert states == -1 and "slice of row" in fault


def test_waits_that_are_skipped_after_one_is_given_up_would_be_found(library):
    """Warps A that no longer waited for their last row would signal the workers twice."""
    states, fault = explore(library, 4, 0, library.grad_barriers(), True, True)
    assert states == -1 and "ready(2)" in fault
