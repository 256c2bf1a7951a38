"""The serving operators' entry points refuse bad arguments on the host,
before any CUDA work (no GPU needed: none of these calls reaches a kernel),
and their plain test implementations agree with hand-worked examples."""
import ctypes
import math

import numpy as np
import pytest

import serving_ref as ref


@pytest.fixture(scope="module")
def lib():
    from stream_compaction_device_gb300 import build as b
    b.build()
    from stream_compaction_device_gb300 import _lib
    return _lib.load()


def at(i):
    """A pointer that is never dereferenced; a MiB apart from the others."""
    return ctypes.c_void_p((i + 1) << 20)


def test_sample_refusals(lib):
    from stream_compaction_device_gb300._lib import ERR_INVALID, OK, SAMPLE_SYMBOLS
    for name in SAMPLE_SYMBOLS:
        fn = getattr(lib, name)
        good = [at(0), 4, 100, 100, at(1), 100, at(2), at(3), at(4), at(5), at(6), at(7), None]

        def call(**change):
            args = list(good)
            for k, v in change.items():
                args[int(k[1:])] = v
            return fn(*args)

        assert call(a0=None) == ERR_INVALID                    # no logits
        assert call(a10=None) == ERR_INVALID                   # no output
        assert call(a2=0) == ERR_INVALID                       # no vocabulary
        assert call(a2=(1 << 18) + 1, a3=1 << 19, a5=1 << 19) == ERR_INVALID
        assert call(a3=99) == ERR_INVALID                      # rows overlap
        assert call(a5=99) == ERR_INVALID
        assert call(a1=2**31) == ERR_INVALID
        assert call(a3=2**61) == ERR_INVALID                   # sizes that wrap
        assert call(a0=ctypes.c_void_p((1 << 20) + 1)) == ERR_INVALID
        assert call(a10=ctypes.c_void_p((7 << 20) + 2)) == ERR_INVALID
        assert call(a10=at(11), a11=ctypes.c_void_p((12 << 20) + 4)) == ERR_INVALID   # the outputs overlap
        assert call(a10=ctypes.c_void_p((1 << 20) + 16)) == ERR_INVALID               # output inside the logits
        assert call(a11=at(1)) == ERR_INVALID                                         # output on the noise
        assert call(a1=0) == OK                                # no rows


def test_block_table_refusals(lib):
    from stream_compaction_device_gb300._lib import ERR_INVALID
    good = [at(0), 8, 4, 8, at(1), at(2), 16, at(3), 50, at(4), at(5), at(6), None]

    def call(**change):
        args = list(good)
        for k, v in change.items():
            args[int(k[1:])] = v
        return lib.block_table_extend_i32(*args)

    for i in (0, 4, 5, 7, 9, 10, 11):
        assert call(**{f"a{i}": None}) == ERR_INVALID, i       # a missing buffer
    assert call(a1=7) == ERR_INVALID                           # rows overlap
    assert call(a2=2**31) == ERR_INVALID
    assert call(a3=-1) == ERR_INVALID
    assert call(a6=0) == ERR_INVALID                           # no page size
    assert call(a8=2**31 - 1) == ERR_INVALID
    assert call(a1=2**61) == ERR_INVALID
    assert call(a11=at(4)) == ERR_INVALID                      # the height in place
    assert call(a7=at(0)) == ERR_INVALID                       # the stack on the table
    assert call(a4=ctypes.c_void_p((2 << 20) + 2)) == ERR_INVALID


def test_slot_map_refusals(lib):
    from stream_compaction_device_gb300._lib import ERR_INVALID
    good = [at(0), 8, 4, 8, at(1), at(2), None, 16, 50, at(3), at(4), at(5), at(6), None]

    def call(**change):
        args = list(good)
        for k, v in change.items():
            args[int(k[1:])] = v
        return lib.slot_map_i32(*args)

    for i in (0, 4, 5, 9, 10, 11, 12):
        assert call(**{f"a{i}": None}) == ERR_INVALID, i
    assert call(a7=-16) == ERR_INVALID
    assert call(a8=2**31) == ERR_INVALID
    assert call(a10=ctypes.c_void_p((5 << 20) + 4)) == ERR_INVALID     # 64-bit slots on 4 bytes
    assert call(a9=at(1)) == ERR_INVALID                               # starts on the lengths
    assert call(a11=at(6)) == ERR_INVALID                              # two outputs alike


def test_release_refusals(lib):
    from stream_compaction_device_gb300._lib import ERR_INVALID
    good = [at(0), 8, 4, 8, at(1), at(2), 16, at(3), 50, at(4), at(5), None]

    def call(**change):
        args = list(good)
        for k, v in change.items():
            args[int(k[1:])] = v
        return lib.block_table_release_i32(*args)

    for i in (0, 4, 5, 7, 9, 10):
        assert call(**{f"a{i}": None}) == ERR_INVALID, i
    assert call(a10=at(4)) == ERR_INVALID                      # the height in place
    assert call(a9=at(3)) == ERR_INVALID                       # the height inside the stack
    assert call(a7=at(0)) == ERR_INVALID                       # the stack on the table
    assert call(a6=0) == ERR_INVALID


def test_reference_draw():
    x = np.log(np.array([0.1, 0.4, 0.4, 0.1]))
    one = np.ones(4)
    assert ref.draw(x, None)[0] == {1}                                    # ties: the lowest index
    assert ref.draw(x, one, k=1)[0] == {1}
    assert ref.draw(x, np.array([1, 9, 1, 1.0]))[0] == {2}
    assert ref.draw(x, np.array([1e-9, 9, 1, 1e-9]), p=0.7)[0] == {2}     # the two largest hold 0.8
    assert ref.draw(x, np.array([1e-9, 9, 1, 1e-9]), p=0.3)[0] == {1}
    assert ref.draw(x, np.array([1e-9, 9, 1, 1e-9]), m=0.5)[0] == {2}
    tokens, logprob = ref.draw(x, np.array([1e-9, 9, 9, 9.0]), k=3)
    assert tokens == {0} and math.isclose(logprob(0)[0], math.log(0.1 / 0.9), rel_tol=1e-9)
    assert ref.draw(np.full(3, -math.inf), np.ones(3))[0] == {-1}


def test_reference_tables():
    table = np.full((3, 4), -1, np.int32)
    pages = np.array([10, 11, 12, 13], np.int32)
    granted, left = ref.extend(table, [0, 0, 0], [5, 9, 4], pages, 4, 4)
    assert granted.tolist() == [1, 0, 0] and left == 2 and table[0].tolist() == [13, 12, -1, -1]
    starts, slots, positions, ids = ref.slots(table, [3, 0, 0], [2, 9, 9], 4, 3, [1, 0, 0])
    assert starts.tolist() == [0, 2, 2, 2] and slots.tolist() == [55, 48, -1]
    assert positions.tolist() == [3, 4, -1] and ids.tolist() == [0, 0, -1]
    assert ref.release(table, [5, 0, 0], [1, 1, 0], pages, 2, 4) == 4 and pages.tolist() == [10, 11, 13, 12]
