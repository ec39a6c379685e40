"""New indices of forks and compactions that overlap an input without being it are refused (the C
ABI's host checks: nothing is launched): a compaction's with its indices, a fork's with the reserved
slots, which are read between the writes."""
import ctypes

import pytest

from test_decode_checks import _pool, lib   # noqa: F401

AT = 1 << 20


@pytest.mark.parametrize("shift", [-60, -4, 4, 60])
def test_new_indices_that_overlap_an_input(lib, shift):   # noqa: F811
    p = lambda x: ctypes.c_void_p(x)   # noqa: E731
    far, ws, need = p(AT + (1 << 16)), p(AT + (1 << 18)), lib.sf_state_workspace(64, 16)
    out = p(AT + shift)
    assert lib.sf_state_compact(_pool(slots=64), p(AT), 16, None, out, ws, need, None) == 1
    assert b"overlaps" in lib.sf_last_error()
    # reserved: one byte a slot, 64 of them
    assert lib.sf_state_fork(_pool(slots=64), far, 16, far, 16, p(AT), out, ws, need, None) == 1
    # beside them, and the indices themselves: on to the workspace's check
    assert lib.sf_state_compact(_pool(slots=64), p(AT), 16, None, p(AT), None, 0, None) == 3
    assert lib.sf_state_fork(_pool(slots=64), p(AT), 16, far, 16, None, p(AT), None, 0, None) == 3
    assert lib.sf_state_compact(_pool(slots=5000), p(AT), 16, None, p(AT + 64), None, 0, None) == 3
