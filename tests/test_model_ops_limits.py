"""Sizes that a launch of the model operators' calls cannot hold are refused as
arguments, and index arithmetic at the largest counts stays in range: on the
host (no call here reaches a kernel)."""
import ctypes
import subprocess

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


SEARCH = """
#include <cstdio>
#include <cstdlib>
#define __host__
#define __device__
#define __forceinline__ inline
#include "search.cuh"
int main(int argc, char **argv)
{
    const long long count = atoll(argv[1]);
    for (int a = 2; a < argc; ++a) {
        const long long answer = atoll(argv[a]);   // places below it come before
        long long wrong = 0;
        auto before = [&](long long i) { wrong += i < 0 || i >= count; return i < answer; };
        const long long one = devscan::first_not(static_cast<int>(count), [&](int i) { return before(i); });
        devscan::Probes p = {0, static_cast<int>(count)};
        int turns = 0;
        while (p.lo < p.hi && ++turns < 64) {
            int many = 0;
            for (int i = 0; i < 32; ++i) many += p.place(i) < p.hi && before(p.place(i));
            p.narrow(many);
        }
        const long long most = answer < count ? answer : count;
        printf("%lld %d\\n", wrong, one == most && p.lo == most && turns < 64);
    }
}
"""


@pytest.fixture(scope="module")
def search(tmp_path_factory):
    """The searches over places below an answer, as a program of the host's."""
    from stream_compaction_device_gb300.build import CSRC
    source = tmp_path_factory.mktemp("search") / "search.cpp"
    source.write_text(SEARCH)
    program = source.with_suffix("")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-I", CSRC, str(source), "-o", str(program)], check=True)
    return str(program)


@pytest.mark.parametrize("count", [0, 1, 2, 31, 32, 33, 1000, 1025, 2**30 + 7, 2**31 - 33, 2**31 - 2, 2**31 - 1])
def test_searches_over_all_rows_that_a_call_takes(search, count):
    """The recurrence's searches for a token's row and a span's first row look at
    no place outside 0 .. count - 1, up to the starts of INT32_MAX - 1 rows."""
    answers = sorted({max(0, min(count, a)) for a in (0, 1, 31, 32, 33, count // 2, count // 3 * 2, count - 33, count - 1, count)})
    told = subprocess.run([search, str(count), *map(str, answers)], check=True, capture_output=True, text=True).stdout.split("\n")
    assert told[: len(answers)] == ["0 1"] * len(answers)
