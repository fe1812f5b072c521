"""Every variant of the attention kernel by its type, head dimension and form,
against the float64 oracle, and units that hundreds of CTAs share."""
from __future__ import annotations

import pytest

from paged_util import PagedCase
from test_gpu_paged import _holes, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    import torch
    from speculative_decoding_verification_25_gb300 import build as b
    b.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _form(c):
    """The host's choice: more than 128 query rows of a key head per request are wide."""
    return "wide" if c.T * (c.Hq // c.Hk) > 128 * max(1, len(c.rows)) else "narrow"


# rows, Hq, Hk, page
SHAPES = {
    "narrow": {
        "tokens": (_rows(31, 50, 2600, 1), 32, 8, 16),
        "drafts": (_holes(_rows(32, 60, 1900, 6)), 24, 4, 32),
        "edges": ([(L, min(L, 3)) for L in (1, 2, 7, 8, 9, 63, 64, 65, 66, 127, 128, 129, 130, 191, 193)], 6, 2, 8),
        "split": ([(15013, 2), (70, 1)], 8, 1, 64),
    },
    "wide": {
        "requests": (_rows(33, 40, 1500, 80), 16, 4, 32),
        "ragged": (_holes(_rows(34, 37, 1200, 167)), 14, 2, 8),
        "edges": ([(L, min(L, 70)) for L in (70, 127, 128, 129, 130, 255, 256, 257, 258, 300, 385)], 12, 3, 16),
        "prompt": ([(1111, 1111), (130, 130)], 4, 2, 128),
        "split": ([(7003, 200)], 6, 1, 64),
    },
}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("form,shape", [(f, s) for f in SHAPES for s in SHAPES[f]])
def test_every_variant(form, shape, D, dtype):
    rows, Hq, Hk, page = SHAPES[form][shape]
    c = PagedCase(rows, Hq, Hk, D, page, dtype, seed=len(shape) + D)
    assert _form(c) == form
    c.check(c.run())


@pytest.mark.parametrize("rows,form,D", [
    ([(40001, 1)], "narrow", 128), ([(32773, 5)], "narrow", 128), ([(20016, 16)], "narrow", 128),
    ([(24015, 15)], "narrow", 64), ([(32832, 64)], "wide", 128), ([(20031, 31)], "wide", 64)])
def test_one_request_on_one_key_head(rows, form, D):
    """What a device that holds one key head sees: one unit cut into up to 304 parts."""
    import torch
    c = PagedCase(rows, 8, 1, D, 64, "bf16", seed=D)
    assert _form(c) == form
    first = c.run()
    c.check(first)
    for _ in range(5):
        r = c.run()
        assert torch.equal(r.out.view(torch.int16), first.out.view(torch.int16)) and torch.equal(r.lse, first.lse)
