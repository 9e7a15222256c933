"""The chunk attention's scratch on the host: how it grows, what is freed and what is kept
(td_chunks.cpp with stand-ins for the CUDA runtime, tests/chunk_host.cpp)."""
from __future__ import annotations

import ctypes as C

import pytest

from tests.test_chunks_host import Call, lib, td


@pytest.fixture
def held(lib):
    """Bytes and buffers held since the test began."""
    lib.fake_held.restype = C.c_int64
    lib.fake_room.argtypes = [C.c_int64]
    bytes0, buffers0 = lib.fake_held(), lib.fake_buffers()
    yield lambda: (lib.fake_held() - bytes0, lib.fake_buffers() - buffers0)
    lib.fake_state(0, 0, 0)
    lib.fake_room(2**62)
    lib.fake_wait(0)


TOKENS = [[(i, 9000, 1) for i in range(n)] for n in (1, 2, 3, 5, 8)]


def test_outgrown_buffers_that_no_capture_used_are_freed(td, lib, held):
    call = Call(td, lib, H=2, D=128)
    for chunks in TOKENS:
        assert call.run("attend", chunks=chunks, nq=14) == td.TD_OK
        assert held() == (4 * lib.fake_floats(), 1)
    before = held()
    for chunks in TOKENS:                                     # nothing grows any more
        assert call.run("attend", chunks=chunks, nq=14) == td.TD_OK
    assert held() == before


def test_a_buffer_that_a_captured_call_used_is_kept(td, lib, held):
    call = Call(td, lib, H=2, D=128)
    assert call.run("attend", chunks=TOKENS[0], nq=14) == td.TD_OK
    kept = held()[0]
    lib.fake_state(0, 1, 0)
    assert call.run("attend", chunks=[(0, 5, 1)], nq=14) == td.TD_OK      # needs none of it
    assert call.run("attend", chunks=TOKENS[0], nq=14) == td.TD_OK
    lib.fake_state(0, 0, 0)
    for i, chunks in enumerate(TOKENS[1:]):
        assert call.run("attend", chunks=chunks, nq=14) == td.TD_OK
        assert held() == (kept + 4 * lib.fake_floats(), 2)


def test_a_captured_call_without_scratch_keeps_nothing(td, lib, held):
    call = Call(td, lib, H=2, D=128)
    assert call.run("attend", chunks=TOKENS[0], nq=14) == td.TD_OK
    lib.fake_state(0, 1, 0)
    assert call.run("attend", chunks=[(0, 5, 1)], nq=14) == td.TD_OK
    lib.fake_state(0, 0, 0)
    assert call.run("attend", chunks=TOKENS[4], nq=14) == td.TD_OK
    assert held() == (4 * lib.fake_floats(), 1)


def test_large_scratch_does_not_double(td, lib, held):
    """A need of 0.9 GB, then a little more: at most 2^28 bytes over it."""
    need = []
    for t in (56000, 60000):
        one = Call(td, lib, H=8, D=128)
        assert one.run("attend8", chunks=[(0, 0, t)], nq=8, layers=(0, 3)) == td.TD_OK
        need.append(4 * lib.fake_floats())
    base = held()
    call = Call(td, lib, H=8, D=128)
    assert call.run("attend8", chunks=[(0, 0, 56000)], nq=8, layers=(0, 3)) == td.TD_OK
    assert held() == (base[0] + need[0], base[1] + 1)
    assert call.run("attend8", chunks=[(0, 0, 60000)], nq=8, layers=(0, 3)) == td.TD_OK
    got, buffers = held()
    assert need[1] <= got - base[0] <= need[1] + 2**28 and buffers == base[1] + 1


def test_a_failed_wait_or_allocation_leaves_a_context_that_works(td, lib, held):
    call = Call(td, lib, H=2, D=128)
    assert call.run("attend", chunks=TOKENS[0], nq=14) == td.TD_OK
    lib.fake_wait(1)
    assert call.run("attend", chunks=TOKENS[4], nq=14) == td.TD_ERR_CUDA and lib.fake_launches() == 0
    lib.fake_wait(0)
    lib.fake_state(0, 0, 1)
    assert call.run("attend", chunks=TOKENS[4], nq=14) == td.TD_ERR_CUDA and lib.fake_launches() == 0
    assert held() == (0, 0)
    lib.fake_state(0, 1, 0)                                   # nothing left to capture with
    assert call.run("attend", chunks=TOKENS[0], nq=14) == td.TD_ERR_INVALID_ARG
    lib.fake_state(0, 0, 0)
    assert call.run("attend", chunks=TOKENS[4], nq=14) == td.TD_OK
    assert held() == (4 * lib.fake_floats(), 1)
