"""The attention's grids keep to their workspace, whatever the number of SMs."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """
#include "sv_ranges.h"
extern "C" {
int ctas(int resident, int rows) { return sv::range_ctas(resident, rows); }
long long room() { return sv::kAttnRows; }
int most() { return sv::kAttnMaxCtas; }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    where = tmp_path_factory.mktemp("grids")
    (where / "grids.cpp").write_text(SOURCE)
    csrc = os.path.join(ROOT, "speculative_decoding_verification_25_gb300", "csrc")
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", "-I" + csrc, "-o", str(where / "grids.so"), str(where / "grids.cpp")],
                   check=True)
    lib = ctypes.CDLL(str(where / "grids.so"))
    lib.room.restype = ctypes.c_longlong
    return lib


# CTAs per SM and rows of a unit: over 16 bits narrow and wide, over 4 bits 16, 32, narrow and wide
@pytest.mark.parametrize("per_sm,rows", [(2, 128), (1, 256), (2, 16), (2, 32), (1, 128), (1, 256)])
def test_two_slots_a_cta_fit(lib, per_sm, rows):
    for sms in range(1, 400):
        ctas = lib.ctas(sms * per_sm, rows)
        assert 1 <= ctas <= min(sms * per_sm, lib.most()) and 2 * ctas * rows <= lib.room()
        assert ctas == sms * per_sm or ctas == lib.most() or 2 * (ctas + 1) * rows > lib.room()
