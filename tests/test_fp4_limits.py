"""Limits of the 4-bit attention's arguments that its arithmetic rests on."""
from test_fp4_refusals import N, _attend   # noqa: F401  (N is a fixture)


def test_contexts_past_the_walks_32_bits_are_refused(N):
    """A unit's keys, its cost (768 at most) and two key tiles of 128 stay below 2^31."""
    for page in (8, 16, 256):
        most = (2 ** 31 - 1024) // page
        assert _attend(N, page=page, max_pages=most + 1) == N.SV_ERR_SHAPE
        assert _attend(N, page=page, max_pages=most, q=None) == N.SV_ERR_NULL   # the shape passes
