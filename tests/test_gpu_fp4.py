"""Attention over the 4-bit cache on the GPU against the 64-bit oracle, within the
bounds that oracle/paged_fp4.py derives per output."""
import math

import numpy as np
import pytest

from fp4_util import Fp4Case

pytestmark = pytest.mark.gpu


def _rows(seed, count, ctx, n):
    rng = np.random.default_rng(seed)
    new = rng.integers(1, n + 1, count)
    return [(int(c + m), int(m)) for c, m in zip(rng.integers(0, ctx + 1, count), new)]


def _holes(rows):
    """Finished requests (no token) and failed ones (no key) among the others."""
    return [(L - n, 0) if b % 7 == 3 else (0, n) if b % 7 == 5 else (L, n) for b, (L, n) in enumerate(rows)]


CASES = {
    "one_key": ([(1, 1)], 1, 1, 64, 8, "bf16"),
    "one_token": ([(1000, 1)], 32, 8, 128, 16, "bf16"),
    "one_token_f16": ([(777, 1)], 8, 8, 64, 64, "f16"),
    "tile_edges": ([(L, 1) for L in (1, 7, 8, 9, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257)], 4, 2, 128, 8, "bf16"),
    "tile_edges_long": ([(L, 40) for L in (40, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300)], 8, 2, 128, 16, "f16"),
    "verify": (_rows(1, 20, 700, 5), 16, 4, 128, 16, "bf16"),
    "long_draft": (_rows(2, 9, 900, 17), 64, 8, 128, 32, "bf16"),
    "odd_group": (_rows(3, 11, 500, 60), 21, 3, 64, 8, "f16"),
    "group_5": (_rows(4, 7, 300, 33), 10, 2, 128, 64, "bf16"),
    "group_9": (_rows(4, 7, 300, 3), 18, 2, 64, 64, "bf16"),
    "group_20": (_rows(4, 7, 600, 3), 40, 2, 128, 16, "f16"),
    "group_33": (_rows(4, 5, 300, 4), 33, 1, 128, 64, "bf16"),
    "group_128": (_rows(5, 3, 300, 3), 128, 1, 64, 16, "bf16"),
    "group_100": (_rows(6, 3, 200, 5), 100, 1, 128, 128, "f16"),
    "no_group": (_rows(7, 5, 400, 130), 3, 3, 64, 256, "bf16"),
    "prompt": ([(519, 519)], 8, 2, 128, 16, "bf16"),
    "prompt_64": ([(1025, 1025), (1, 1), (300, 300)], 4, 1, 64, 32, "f16"),
    "chunk": ([(1300, 257), (900, 256)], 8, 1, 128, 128, "bf16"),
    "empty_rows": ([(0, 3), (20, 0), (2, 5), (0, 0), (130, 129), (0, 1), (64, 70)], 6, 2, 128, 8, "bf16"),
    "empty_rows_64": ([(0, 300), (0, 0), (100, 200)], 4, 4, 64, 16, "f16"),
    "all_empty": ([(0, 2), (0, 0)], 2, 1, 64, 8, "bf16"),
    "many": ([(1 + b % 90, 1 + b % 3) for b in range(700)], 2, 1, 64, 8, "bf16"),
    "mixed": ([(2000, 1), (600, 600), (1500, 5), (31, 31), (4000, 1)], 8, 2, 128, 64, "bf16"),
    "many_tiles": (_rows(8, 60, 3000, 5), 16, 8, 128, 16, "bf16"),
    "many_tiles_64": (_rows(9, 150, 2500, 3), 8, 8, 64, 64, "f16"),
    "many_tiles_long": (_rows(10, 40, 1500, 70), 8, 4, 64, 32, "bf16"),
    "ragged_units": (_rows(11, 37, 1500, 167), 14, 2, 64, 8, "f16"),
    "ragged_units_128": (_rows(12, 24, 900, 300), 8, 2, 128, 16, "bf16"),
    "holes": (_holes(_rows(13, 70, 2500, 5)), 32, 8, 128, 32, "bf16"),
    "holes_one_token": (_holes(_rows(14, 105, 400, 1)), 64, 8, 64, 128, "f16"),
    "holes_long": (_holes(_rows(15, 37, 1200, 167)), 14, 2, 64, 8, "f16"),
    "split": ([(20011, 1)], 8, 1, 128, 64, "bf16"),
    "split_long": ([(9000, 300)], 4, 1, 64, 32, "bf16"),
}
GAINS = {"verify": (0.5, 2.0), "odd_group": (0.3, 0.1), "chunk": (4.0, 0.0625)}


@pytest.mark.parametrize("name", CASES)
def test_attention_matches_the_oracle(name):
    import torch
    from speculative_decoding_verification_25_gb300 import _native as N, api
    rows, *shape = CASES[name]
    gains = tuple(float(np.float32(g)) for g in GAINS.get(name, (1.0, 1.0)))
    c = Fp4Case(rows, *shape, seed=len(name), gains=gains)
    c.check(c.run())
    counters = api.attention_workspace(c.D, torch.device("cuda:0"))[:N.SV_ATTENTION_COUNTER_BYTES]
    assert int(counters.sum()) == 0     # ready for the next call


@pytest.mark.parametrize("spread", [0.02, 4.0])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attention_of_flat_and_of_peaked_scores(spread, dtype):
    """Scores near zero, and scores of +-100 whose maximum keeps moving."""
    c = Fp4Case([(700, 3), (90, 90)], 8, 2, 128, 16, dtype, seed=11, spread=spread)
    c.check(c.run())


def test_attention_of_rising_scores():
    """Every tile brings a new maximum, first by much and then by little."""
    import torch
    c = Fp4Case([(1600, 2), (1513, 129)], 4, 1, 64, 8, "bf16", seed=5)
    for b, (L, n) in enumerate(c.rows):
        k = (torch.sqrt(torch.arange(L, dtype=torch.float64))[:, None, None] * torch.ones(L, 1, 64) / 8).to(torch.bfloat16)
        c.host[b][0] = k.double().numpy()
        ids = c.block_table[b, :-(-L // 8)].long()
        padded = torch.full((len(ids) * 8, 1, 64), float("nan"), dtype=torch.bfloat16)
        padded[:L] = k
        c.k_cache[ids] = padded.view(-1, 8, 1, 64).transpose(1, 2).to("cuda:0")
    c.encode()
    c.qkv.abs_()
    c.check(c.run())


@pytest.mark.parametrize("factor", [2.0 ** -100, 2.0 ** 60, 2.0 ** 100])
def test_attention_of_queries_outside_the_range_of_float16(factor):
    """bfloat16 queries of any size, rows of one unit that differ by far among them."""
    c = Fp4Case([(700, 3), (90, 90)], 8, 2, 128, 16, "bf16", seed=17)
    c.qkv.mul_(factor)
    c.qkv[::3] *= 2.0 ** -20
    c.scale = float(np.float32(c.scale / factor))
    c.check(c.run())


def test_attention_of_plain_q_and_of_padded_tokens():
    c = Fp4Case([(300, 4), (50, 7)], 8, 2, 64, 16, "bf16", seed=3, qkv=False, extra_tokens=9)
    r = c.run()
    c.check(r)
    assert float(r.out[11:].abs().sum()) == 0 and bool((r.lse[11:] == -math.inf).all())


def test_attention_of_no_requests():
    c = Fp4Case([], 4, 2, 64, 8, "bf16", extra_tokens=3)
    r = c.run()
    assert float(r.out.abs().sum()) == 0 and bool((r.lse == -math.inf).all())
    assert Fp4Case([(4, 0)], 4, 2, 64, 8, "bf16").run().out.shape == (0, 4, 64)


def test_attention_past_32_bit_offsets():
    """Codes of more than 2^32 bytes, the requests on the last pages."""
    import torch
    from speculative_decoding_verification_25_gb300 import api
    c = Fp4Case([(3000, 2), (700, 300)], 8, 4, 128, 16, "bf16", seed=9)
    small, n = c.cache, c.cache.k.shape[0]
    far = 2 ** 32 // (4 * 16 * 64) + 400 - n
    parts = []
    for t in small:
        big = torch.empty(far + n, *t.shape[1:], dtype=torch.uint8, device=t.device)
        big[far:] = t.view(torch.uint8)
        parts.append(big.view(t.dtype))
    c.cache = api.PagedCacheFp4(*parts)
    c.block_table = torch.where(c.block_table < n, c.block_table + far, c.block_table)
    assert c.cache.k.numel() > 2 ** 32
    c.check(c.run())


def test_attention_flags_bad_lengths_and_pages():
    import torch
    from speculative_decoding_verification_25_gb300 import _native as N
    flags = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    c = Fp4Case([(40, 2), (70, 3), (30, 1)], 4, 2, 64, 16, "bf16", seed=2)
    good = c.run(flags=flags)
    assert flags.item() == 0
    # a page outside the cache reads as zeros: its scores are 0, its values add nothing
    c.block_table[1, 0] = c.cache.k.shape[0]
    r = c.run(flags=flags)
    assert flags.item() == N.SV_DEV_BAD_PAGE
    c.host[1][:, :16] = 0
    c.check(r)
    flags.zero_()
    c.block_table[1, 0] = -1
    c.check(c.run(flags=flags))
    assert flags.item() == N.SV_DEV_BAD_PAGE
    # lengths outside the table are clamped, the other rows stay what they are
    flags.zero_()
    c.kv_len[1] = -3
    r = c.run(flags=flags)
    assert flags.item() == N.SV_DEV_BAD_LENGTH
    assert float(r.out[2:5].abs().sum()) == 0
    torch.testing.assert_close(r.out[[0, 1, 5]], good.out[[0, 1, 5]], rtol=0, atol=0)
    # offsets that decrease: the row is skipped
    flags.zero_()
    c.kv_len[1] = 0
    c.cu_new.copy_(torch.tensor([0, 2, 1, 6]))
    c.run(flags=flags)
    assert flags.item() & N.SV_DEV_BAD_LENGTH


@pytest.mark.parametrize("name", ["verify", "many_tiles", "many_tiles_64", "ragged_units", "ragged_units_128", "mixed",
                                  "split", "split_long", "empty_rows"])
def test_attention_gives_the_same_bits_every_time(name):
    import torch
    rows, *shape = CASES[name]
    c = Fp4Case(rows, *shape, seed=1)
    first = c.run()
    for _ in range(20):
        r = c.run()
        assert torch.equal(r.out.view(torch.int16), first.out.view(torch.int16)) and torch.equal(r.lse, first.lse)


def test_attention_on_two_streams_at_once():
    import torch
    cases = [Fp4Case([(5000, 1), (100, 40)], 8, 2, 128, 16, "bf16", seed=s) for s in (1, 2)]
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[c.run(stream=s) for c, s in zip(cases, streams)] for _ in range(30)]
    torch.cuda.synchronize()
    for pair in got:
        for r, w in zip(pair, want):
            assert torch.equal(r.out, w.out) and torch.equal(r.lse, w.lse)


def test_attention_of_scores_and_values_that_are_not_finite():
    """A NaN query row is NaN alone; a NaN key is NaN where it is seen; an infinite
    query row's scores are infinite or NaN and leave the other rows alone."""
    import torch
    c = Fp4Case([(300, 40), (200, 1)], 4, 2, 64, 16, "bf16", seed=6)
    good = c.run()
    c.qkv[5, 1] = float("nan")
    c.qkv[7, 2, 3] = float("inf")
    r = c.run()
    assert bool(r.out[5, 1].isnan().all()) and bool(r.lse[5, 1].isnan())
    assert bool(r.out[7, 2].isnan().all()) and bool(r.lse[7, 2].isnan())
    r.out[5, 1], r.lse[5, 1] = good.out[5, 1], good.lse[5, 1]
    r.out[7, 2], r.lse[7, 2] = good.out[7, 2], good.lse[7, 2]
    # rows of the same unit share the power of two that queries are scaled by
    torch.testing.assert_close(r.out, good.out, rtol=2.0 ** -7, atol=1e-6)
    c = Fp4Case([(300, 40), (200, 1)], 4, 2, 64, 16, "bf16", seed=6)
    page, off = int(c.block_table[0, 280 // 16]), 280 % 16
    c.cache.k_scale.view(torch.uint8)[page, 1, off, 2] = 127     # key 280 of key head 1
    r = c.run()
    seen = torch.arange(40, device="cuda:0") >= 280 - 260        # tokens that see it
    assert bool(r.out[:40][seen][:, 2:].isnan().all()) and bool(r.lse[:40][seen][:, 2:].isnan().all())
    assert torch.equal(r.out[:40][seen][:, :2], good.out[:40][seen][:, :2])
    assert torch.equal(r.out[:40][~seen], good.out[:40][~seen]) and torch.equal(r.out[40:], good.out[40:])
