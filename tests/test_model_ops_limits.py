"""Sizes that a launch of the model operators' calls cannot hold are refused as
arguments, and index arithmetic at the largest counts stays in range: on the
host (no call here reaches a kernel)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from stream_compaction_device_gb300 import build as b
    b.build()
    from stream_compaction_device_gb300 import _lib
    return _lib.load()


def at(i):
    """A pointer that is never dereferenced, 2^42 bytes apart from the others."""
    return ctypes.c_void_p((i + 1) << 42)


def test_more_tokens_and_rows_than_a_grid_has_blocks(lib):
    from stream_compaction_device_gb300 import _lib
    most = 2**31 - 1
    for tokens, rows in ((most, 1), (most, most), (most - 100, 900), (2**31 - 2**28 + 1, most)):
        assert lib.expert_dispatch(at(0), 16, 16, tokens, 1, at(1), rows, at(2), at(3), 16, None) == _lib.ERR_INVALID
    for tokens, rows in ((most, 1), (most, most), (most - 100, 3500), (2**31 - 2**26 + 1, most)):
        for name in _lib.EXPERT_COMBINE_BACKWARD_SYMBOLS:
            assert getattr(lib, name)(at(0), 8, at(1), 8, rows, tokens, 1, 8, at(2), at(3), at(4), at(5), 8, at(6), None) == _lib.ERR_INVALID
