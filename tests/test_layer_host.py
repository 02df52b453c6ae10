"""Host checks of the decoder-layer kernels' index arithmetic: headers that
both the kernels and these tests compile (no GPU needed)."""
import ctypes
import itertools
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_mixed_precision_amd", "csrc")
MAX, MIN = 2**31 - 1, -(2**31)


def _compile(tmp, source):
    src, lib = tmp / "host.cpp", tmp / "host.so"
    src.write_text(source)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib))


@pytest.fixture(scope="module")
def rows(tmp_path_factory):
    lib = _compile(tmp_path_factory.mktemp("rows"), """
#include "attn_rows.h"
extern "C" void rows(int start, int end, int total, int most, int *out)
{
    const bq::QueryRows r = bq::query_rows_of(start, end, total, most);
    out[0] = r.first;
    out[1] = r.count;
    out[2] = r.len;
}
""")

    def call(*a):
        out = (ctypes.c_int * 3)()
        lib.rows(*a, out)
        return tuple(out)

    return call


def _cases():
    ends = [MIN, MIN + 1, -2, -1, 0, 1, 2, 7, 8, 9, 100, MAX - 1, MAX]
    yield from itertools.product(ends, ends, [1, 8, 100, 2**30], [1, 3, 8, 2**30])
    rng = random.Random(0)
    for _ in range(2000):
        yield rng.randint(MIN, MAX), rng.randint(MIN, MAX), rng.randint(1, 2**30), rng.randint(1, 2**30)


def test_query_rows_stay_inside_the_queries(rows):
    """Whatever the starts hold, the rows lie in [0, total_q) and are those of
    the range taken within it."""
    for start, end, total, most in _cases():
        first, count, _ = rows(start, end, total, most)
        lo, hi = min(max(start, 0), total), min(max(end, 0), total)
        assert 0 <= first and 0 <= count and first + count <= total, (start, end, total, most, first, count)
        assert count == min(max(hi - lo, 0), most), (start, end, total, most)
        assert count == 0 or first == lo


def test_query_positions_do_not_depend_on_the_most_computed(rows):
    """The length that positions are counted from is the whole range's."""
    for start, end, total, most in _cases():
        first, count, length = rows(start, end, total, most)
        lo, hi = min(max(start, 0), total), min(max(end, 0), total)
        assert length == max(hi - lo, 0) and count == min(length, most), (start, end, total, most)
