"""The arithmetic that cuts the attention's work into ranges, compiled for the
host, at sizes past 31 and 32 bits."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """
#include "sv_ranges.h"
extern "C" {
long long quota(long long total, unsigned ctas, int least) { return sv::range_quota(total, ctas, least); }
int back(int pos, long long quota) { return sv::ranges_back(pos, quota); }
int ahead(long long at, long long quota) { return sv::ranges_ahead(at, quota); }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    where = tmp_path_factory.mktemp("ranges")
    (where / "ranges.cpp").write_text(SOURCE)
    csrc = os.path.join(ROOT, "speculative_decoding_verification_25_gb300", "csrc")
    subprocess.run(["g++", "-O1", "-fwrapv", "-shared", "-fPIC", "-I" + csrc, "-o", str(where / "ranges.so"),
                    str(where / "ranges.cpp")], check=True)
    lib = ctypes.CDLL(str(where / "ranges.so"))
    lib.quota.restype, lib.quota.argtypes = ctypes.c_longlong, [ctypes.c_longlong, ctypes.c_uint, ctypes.c_int]
    lib.back.argtypes, lib.ahead.argtypes = [ctypes.c_int, ctypes.c_longlong], [ctypes.c_longlong] * 2
    return lib


def _totals(ctas):
    near = [0, 1, 64, ctas, 2 ** 31, 2 ** 32 - ctas, 2 ** 32 - 1, 2 ** 32, 2 ** 32 + ctas, ctas << 32, 2 ** 45]
    rng = np.random.default_rng(ctas)
    return [t + d for t in near for d in (-2, -1, 0, 1, 2) if t + d >= 0] + \
           [int(2 ** x) for x in rng.uniform(0, 50, 200)]


@pytest.mark.parametrize("ctas,least", [(1, 64), (152, 128), (160, 128), (304, 64), (320, 64)])
def test_ranges_cover_the_work_evenly(lib, ctas, least):
    for total in _totals(ctas):
        assert lib.quota(total, ctas, least) == max(least, -(-total // ctas)), total


@pytest.mark.parametrize("quota", [64, 100, 128, 4099, 2 ** 30, 2 ** 31 - 1, 2 ** 31 + 5, 2 ** 32 - 1, 2 ** 32, 2 ** 33 + 1])
def test_first_and_last_range_of_a_unit(lib, quota):
    top = 2 ** 31 - 1
    for pos in {0, 1, 63, 64, 65, 10 ** 6, 2 ** 30, 2 ** 30 + 1, top - 1, top,
                *(min(top, max(0, quota * k + d)) for k in (1, 2) for d in (-1, 0, 1))}:
        assert lib.back(pos, quota) == -(-pos // quota), pos
    for at in (0, 1, quota - 1, quota, 7 * quota - 1, 7 * quota, 319 * quota + 5, 2 ** 31, 2 ** 32 - 1, 2 ** 32):
        assert lib.ahead(at, quota) == at // quota, at
