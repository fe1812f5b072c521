"""paged_attention of NaN and infinite scores: a row that sees one is NaN in
out and in lse (never "sees no key"), and the rows beside it keep their bits."""
from __future__ import annotations

import pytest

from paged_util import PagedCase

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
# whole units and units that several CTAs join; the last token's row is spoilt
SHAPES = {
    "narrow": ([(70, 3), (300, 2)], 8, 2, 128, 16, "bf16"),
    "narrow_split": ([(20011, 1), (64, 1)], 8, 1, 128, 64, "f16"),
    "wide": ([(300, 300), (90, 90)], 4, 2, 64, 8, "f16"),
    "wide_split": ([(9000, 300)], 4, 1, 128, 32, "bf16"),
}


@pytest.fixture(scope="module", autouse=True)
def library():
    import torch
    from speculative_decoding_verification_25_gb300 import build as b
    b.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _compare(got, clean, spoilt):
    """`spoilt` [T, Hq]: the rows that see the value; the others keep their bits."""
    import torch
    assert bool(got.out[spoilt].isnan().all()) and bool(got.lse[spoilt].isnan().all())
    assert torch.equal(got.out[~spoilt], clean.out[~spoilt]) and torch.equal(got.lse[~spoilt], clean.lse[~spoilt])


@pytest.mark.parametrize("name", SHAPES)
def test_nan_in_a_query(name):
    import torch
    rows, *shape = SHAPES[name]
    c = PagedCase(rows, *shape, seed=3)
    clean = c.run()
    c.q[c.T - 1, 2, 5] = NAN
    spoilt = torch.zeros(c.T, c.Hq, dtype=torch.bool, device="cuda:0")
    spoilt[c.T - 1, 2] = True
    _compare(c.run(), clean, spoilt)


@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("name", SHAPES)
def test_a_key_that_spoils_its_scores(name, value):
    """The last key of the first request, which only its last token sees: the
    tokens before mask it.  An infinite key of one sign with queries of that
    sign has the score +inf; with the other sign -inf, a probability of 0."""
    import torch
    rows, *shape = SHAPES[name]
    c = PagedCase(rows, *shape, seed=4)
    L, n = rows[0]
    c.q[:, :, 7].abs_().add_(0.5)
    clean = c.run()
    page = int(c.block_table[0, (L - 1) // c.page])
    c.k_cache[page, 0, (L - 1) % c.page, 7] = value
    G = c.Hq // c.Hk
    spoilt = torch.zeros(c.T, c.Hq, dtype=torch.bool, device="cuda:0")
    spoilt[n - 1, :G] = True
    _compare(c.run(), clean, spoilt)


def test_scores_of_minus_infinity_count_as_masked():
    """Every key -inf: the row's sum is empty."""
    import torch
    c = PagedCase([(40, 1)], 2, 2, 64, 8, "bf16", seed=6)
    c.q[:, :, 7] = 1.0
    for p in c.block_table[0, :5].tolist():
        c.k_cache[p, 0, :, 7] = -INF
    r = c.run()
    assert bool((r.lse[:, 0] == -INF).all()) and float(r.out[:, 0].abs().sum()) == 0
    assert bool(r.lse[:, 1].isfinite().all())
