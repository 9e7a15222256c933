"""td_update_tables' index arithmetic at the ends of its ranges, on the host (tests/tables_host.cpp)."""
from __future__ import annotations

import ctypes as C
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    from collective_kv_cache_gb300 import build
    out = str(tmp_path_factory.mktemp("tables_host") / "libtables_host.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-Wall", "-I", build.INC, "-I",
                    build.CSRC, "-I", os.path.join(build.CUDA_HOME, "include"),
                    os.path.join(ROOT, "tests", "tables_host.cpp"), "-o", out], check=True)
    h = C.CDLL(out)
    h.host_tables_grid.restype = C.c_int64
    h.host_tables_goes_on.argtypes = [C.c_int64] * 3
    return h


@pytest.mark.parametrize("sms", [8, 152])
@pytest.mark.parametrize("P", [1, 16, 2 ** 30])
@pytest.mark.parametrize("max_slots", [0, 1, 100000, 2 ** 30, MOST - 1, MOST])
@pytest.mark.parametrize("n", [0, 1, 4096])
def test_the_grid_is_in_its_limits(lib, n, max_slots, P, sms):
    want = max((max_slots // P + n) // 256 + 1, n // 2 + 1)
    assert lib.host_tables_grid(n, P, max_slots, sms) == min(want, 4 * sms)


@pytest.mark.parametrize("end", [MOST, MOST - 1, 2 ** 31 - 155648, 2 ** 30, 1000])
def test_no_index_is_below_the_end_again_once_it_has_passed_it(lib, end):
    """A thread's last place below the end, and the step of the largest grid from there; the loops over
    pages and slots begin at up to the end plus a thread's number."""
    step = 4 * 152 * 256
    for thread in (0, 1, 31, 255, 1000, step // 2, step - 1):
        first = thread if thread < end else None
        if first is not None:
            last = thread + (end - 1 - thread) // step * step
            assert not lib.host_tables_goes_on(last, step, end)
        assert not lib.host_tables_goes_on(end, thread, end)


@pytest.mark.parametrize("P", [1, 3, 16, 2 ** 30 - 1, 2 ** 30, 2 ** 30 + 1, MOST - 1, MOST])
def test_pages_of_the_longest_requests_and_the_largest_pages(lib, P):
    for length in (0, 1, 2, 5, 16, 2 ** 30 - 2, 2 ** 30 - 1):
        assert lib.host_pages_of(length, P) == -(-length // P)
