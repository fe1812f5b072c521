"""The paged cache operators on the GPU against the 64-bit oracle: plans are
equal entry by entry, appended caches bit by bit, attention within the bounds
that oracle/paged.py derives per output."""
import math

import numpy as np
import pytest

from oracle import paged as oracle
from paged_util import PagedCase, torch_dtype

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ plan

def _device(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to("cuda:0")


def _run_plan(seq, new, held, table, stack, n_pages, page, max_tokens, in_place=False):
    import torch
    from speculative_decoding_verification_25_gb300 import api
    free = np.full(n_pages, -5, np.int32)
    free[:len(stack)] = stack
    t = dict(seq=_device(seq), new=_device(new), held=_device(held), table=_device(table), free=_device(free),
             count=_device([len(stack)]))
    flags = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    out = None
    if in_place:
        e = lambda n: torch.empty(n, dtype=torch.int32, device="cuda:0")
        out = api.PagedPlan(e(len(seq) + 1), e(len(seq)), e(max_tokens), e(max_tokens), t["held"], t["count"])
    p = api.paged_plan(t["seq"], t["new"], t["held"], t["table"], t["free"], t["count"], page_size=page,
                       max_tokens=max_tokens, out=out, flags=flags)
    torch.cuda.synchronize()
    return p, t, int(flags.item())


def _compare_plan(got, t, ref):
    np.testing.assert_array_equal(got.cu_new.cpu().numpy(), ref.cu_new)
    np.testing.assert_array_equal(got.kv_len.cpu().numpy(), ref.kv_len)
    np.testing.assert_array_equal(got.slot_map.cpu().numpy(), ref.slot_map)
    np.testing.assert_array_equal(got.positions.cpu().numpy(), ref.positions)
    np.testing.assert_array_equal(got.page_count.cpu().numpy(), ref.page_count)
    np.testing.assert_array_equal(t["table"].cpu().numpy(), ref.block_table)
    n = int(got.free_count.item())
    assert n == len(ref.stack)
    np.testing.assert_array_equal(t["free"].cpu().numpy()[:n], ref.stack)


def _plan_state(rng, B, page, width, n_max, broken=False):
    cap = width * page
    seq = rng.integers(0, max(1, cap - n_max) + 1, B)
    new = np.minimum(rng.integers(0, n_max + 1, B), cap - seq)
    held = np.minimum(-(-seq // page) + rng.integers(0, 4, B) * (rng.random(B) < 0.4), width)
    done = rng.random(B) < 0.1
    seq[done], new[done] = 0, 0
    pages = rng.permutation(int(held.sum()) + int((-(-(seq + new) // page)).sum()) + 3)
    table = rng.integers(0, 3, (B, width))
    at = 0
    for b in range(B):
        table[b, :held[b]] = pages[at:at + held[b]]
        at += held[b]
    if broken and B > 6:
        seq[1], new[2], held[3], held[4] = -1, -4, -2, width + 1
        seq[5], new[5] = cap, 1
    return seq, new, held, table, pages[at:], len(pages)


@pytest.mark.parametrize("B,page,width,n_max", [
    (1, 16, 9, 5), (2, 8, 3, 1), (31, 8, 40, 17), (64, 16, 70, 5), (300, 256, 5, 700), (1023, 32, 33, 40),
    (1024, 64, 4, 3), (1025, 8, 9, 20), (2500, 16, 6, 9), (8192, 8, 4, 2), (3, 128, 600, 60000), (5, 8, 2000, 9999)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_matches_the_oracle(B, page, width, n_max, in_place):
    rng = np.random.default_rng(B * page)
    seq, new, held, table, stack, n_pages = _plan_state(rng, B, page, width, n_max)
    total = int(new.sum())
    got, t, flags = _run_plan(seq, new, held, table, stack, n_pages, page, total + B % 3, in_place)
    ref = oracle.plan(seq, new, held, table.astype(np.int32), stack, page, total + B % 3)
    _compare_plan(got, t, ref)
    assert flags == 0


@pytest.mark.parametrize("B,page,width,n_max", [(7, 8, 5, 9), (64, 16, 20, 33), (1500, 8, 8, 11)])
@pytest.mark.parametrize("short", ["pages", "tokens", "both", "none"])
def test_plan_of_rows_that_cannot_be_served(B, page, width, n_max, short):
    from speculative_decoding_verification_25_gb300 import _native as N
    rng = np.random.default_rng(B + len(short))
    seq, new, held, table, stack, n_pages = _plan_state(rng, B, page, width, n_max, broken=True)
    ok = (seq >= 0) & (new >= 0)
    max_tokens = int(new[ok].sum()) // (2 if short in ("tokens", "both") else 1) + 1
    if short in ("pages", "both"):
        stack = stack[:len(stack) // 5]
    ref = oracle.plan(seq, new, held, table.astype(np.int32), stack, page, max_tokens)
    got, t, flags = _run_plan(seq, new, held, table, stack, n_pages, page, max_tokens)
    _compare_plan(got, t, ref)
    assert bool(flags & N.SV_DEV_NO_PAGES) == ref.no_pages
    assert bool(flags & N.SV_DEV_TOKENS_CLIPPED) == ref.clipped
    assert bool(flags & N.SV_DEV_BAD_LENGTH) == ref.bad_length


def test_plan_of_no_rows_and_of_no_tokens():
    got, t, flags = _run_plan([], [], [], np.zeros((0, 3)), [4, 2], 5, 16, 6)
    assert got.cu_new.tolist() == [0] and got.slot_map.tolist() == [-1] * 6 and got.free_count.tolist() == [2]
    got, t, flags = _run_plan([5, 0], [0, 0], [1, 1], np.array([[3, 0], [1, 0]]), [4, 2], 5, 16, 0)
    assert got.cu_new.tolist() == [0, 0, 0] and got.kv_len.tolist() == [5, 0]
    assert got.page_count.tolist() == [1, 0] and t["free"].tolist()[:3] == [4, 2, 1] and flags == 0


def test_plan_flags_pages_outside_the_cache():
    from speculative_decoding_verification_25_gb300 import _native as N
    got, t, flags = _run_plan([3, 3], [2, 2], [1, 1], np.array([[99], [2]]), [4], 5, 16, 4)
    assert got.slot_map.tolist() == [-1, -1, 35, 36] and flags == N.SV_DEV_BAD_PAGE


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("T,Hk,D,page,dtype", [
    (1, 1, 64, 8, "bf16"), (5, 8, 128, 16, "bf16"), (333, 3, 64, 32, "f16"), (2049, 8, 128, 256, "f16"),
    (7001, 5, 128, 64, "bf16"), (40000, 1, 64, 128, "bf16")])
def test_append_is_bit_exact(T, Hk, D, page, dtype):
    import torch
    from speculative_decoding_verification_25_gb300 import api
    g = torch.Generator().manual_seed(T)
    dt = torch_dtype(dtype)
    n_pages = -(-T // page) + 3
    bits = lambda *s: torch.randint(-2 ** 15, 2 ** 15, s, generator=g).to(torch.int16)   # any bits, NaN among them
    new, k, v = bits(T, 2 * Hk + 1, D), bits(n_pages, Hk, page, D), bits(n_pages, Hk, page, D)
    slots = torch.randperm(n_pages * page, generator=g)[:T].to(torch.int32)
    slots[::7] = -1
    want = oracle.append(new[:, :Hk].numpy(), new[:, Hk + 1:].numpy(), slots.numpy(), k.numpy(), v.numpy())
    d = new.to("cuda:0").view(dt)
    kd, vd = k.to("cuda:0").view(dt), v.to("cuda:0").view(dt)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    api.paged_append(d[:, :Hk], d[:, Hk + 1:], slots.to("cuda:0"), kd, vd, flags=flags)
    np.testing.assert_array_equal(kd.view(torch.int16).cpu().numpy(), want[0])
    np.testing.assert_array_equal(vd.view(torch.int16).cpu().numpy(), want[1])
    assert flags.item() == 0


def test_append_skips_slots_past_the_cache():
    import torch
    from speculative_decoding_verification_25_gb300 import _native as N, api
    new = torch.ones(3, 1, 64, dtype=torch.bfloat16, device="cuda:0")
    k, v = (torch.zeros(2, 1, 8, 64, dtype=torch.bfloat16, device="cuda:0") for _ in range(2))
    flags = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    api.paged_append(new, new, _device([15, 16, 2 ** 31 - 1]), k, v, flags=flags)
    assert float(k.sum()) == 64 and float(v[1, 0, 7].sum()) == 64 and flags.item() == N.SV_DEV_BAD_PAGE


# ------------------------------------------------------------- attention

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
    "tile_edges_wide": ([(L, 40) for L in (40, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300)], 8, 2, 128, 16, "f16"),
    "verify": (_rows(1, 20, 700, 5), 16, 4, 128, 16, "bf16"),
    "long_draft": (_rows(2, 9, 900, 17), 64, 8, 128, 32, "bf16"),
    "odd_group": (_rows(3, 11, 500, 60), 21, 3, 64, 8, "f16"),
    "group_5": (_rows(4, 7, 300, 33), 10, 2, 128, 64, "bf16"),
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
    "many_tiles_wide": (_rows(10, 40, 1500, 70), 8, 4, 64, 32, "bf16"),
    "ragged_units": (_rows(11, 37, 1500, 167), 14, 2, 64, 8, "f16"),
    "ragged_units_128": (_rows(12, 24, 900, 300), 8, 2, 128, 16, "bf16"),
    "holes": (_holes(_rows(13, 70, 2500, 5)), 32, 8, 128, 32, "bf16"),
    "holes_one_token": (_holes(_rows(14, 105, 400, 1)), 64, 8, 64, 128, "f16"),
    "holes_wide": (_holes(_rows(15, 37, 1200, 167)), 14, 2, 64, 8, "f16"),
    "holes_wide_128": (_holes(_rows(16, 24, 900, 120)), 16, 4, 128, 64, "bf16"),
    "split": ([(20011, 1)], 8, 1, 128, 64, "bf16"),
    "split_wide": ([(9000, 300)], 4, 1, 64, 32, "bf16"),
}


@pytest.mark.parametrize("name", CASES)
def test_attention_matches_the_oracle(name):
    import torch
    from speculative_decoding_verification_25_gb300 import _native as N, api
    rows, *shape = CASES[name]
    c = PagedCase(rows, *shape, seed=len(name))
    c.check(c.run())
    counters = api.attention_workspace(c.D, torch.device("cuda:0"))[:N.SV_ATTENTION_COUNTER_BYTES]
    assert int(counters.sum()) == 0     # ready for the next call


@pytest.mark.parametrize("spread", [0.02, 4.0])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attention_of_flat_and_of_peaked_scores(spread, dtype):
    """Scores near zero, and scores of +-100 whose maximum keeps moving."""
    c = PagedCase([(700, 3), (90, 90)], 8, 2, 128, 16, dtype, seed=11, spread=spread)
    c.check(c.run())


def test_attention_of_rising_scores():
    """Every tile brings a new maximum, first by much and then by little."""
    import torch
    c = PagedCase([(600, 2), (513, 129)], 4, 1, 64, 8, "bf16", seed=5)
    for b, (L, n) in enumerate(c.rows):
        at = torch.arange(L, dtype=torch.float64)
        k = (torch.sqrt(at)[:, None, None] * torch.ones(L, 1, 64) / 8).to(torch.bfloat16)
        c.host[b][0] = k.double().numpy()
        ids = c.block_table[b, :-(-L // 8)].long()
        padded = torch.full((len(ids) * 8, 1, 64), float("nan"), dtype=torch.bfloat16)
        padded[:L] = k
        c.k_cache[ids] = padded.view(-1, 8, 1, 64).transpose(1, 2).to("cuda:0")
    c.qkv.abs_()
    c.check(c.run())


def test_attention_of_plain_q_and_of_padded_tokens():
    c = PagedCase([(300, 4), (50, 7)], 8, 2, 64, 16, "bf16", seed=3, qkv=False, extra_tokens=9)
    r = c.run()
    c.check(r)
    assert float(r.out[11:].abs().sum()) == 0 and bool((r.lse[11:] == -math.inf).all())


def test_attention_of_no_requests():
    import torch
    c = PagedCase([], 4, 2, 64, 8, "bf16", extra_tokens=3)
    r = c.run()
    assert float(r.out.abs().sum()) == 0 and bool((r.lse == -math.inf).all())
    assert PagedCase([(4, 0)], 4, 2, 64, 8, "bf16").run().out.shape == (0, 4, 64)


def test_attention_past_32_bit_offsets():
    """A cache of 2^31 elements and more, the requests on its last pages."""
    c = PagedCase([(3000, 2), (700, 300)], 8, 8, 128, 16, "bf16", seed=9, n_pages=2 ** 31 // (8 * 128 * 16) + 400)
    assert c.k_cache.numel() > 2 ** 31
    c.check(c.run())


def test_attention_flags_bad_lengths_and_pages():
    import torch
    from speculative_decoding_verification_25_gb300 import _native as N
    flags = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    c = PagedCase([(40, 2), (70, 3), (30, 1)], 4, 2, 64, 16, "bf16", seed=2)
    good = c.run(flags=flags)
    assert flags.item() == 0
    # a page outside the cache reads as zeros: its scores are 0, its values add nothing
    c.block_table[1, 0] = c.k_cache.shape[0]
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


@pytest.mark.parametrize("name", ["verify", "many_tiles", "many_tiles_64", "ragged_units",
                                  "ragged_units_128", "mixed", "split", "split_wide", "empty_rows"])
def test_attention_gives_the_same_bits_every_time(name):
    import torch
    rows, *shape = CASES[name]
    c = PagedCase(rows, *shape, seed=1)
    first = c.run()
    for _ in range(20):
        r = c.run()
        assert torch.equal(r.out.view(torch.int16), first.out.view(torch.int16)) and torch.equal(r.lse, first.lse)


def test_attention_on_two_streams_at_once():
    import torch
    cases = [PagedCase([(5000, 1), (100, 40)], 8, 2, 128, 16, "bf16", seed=s) for s in (1, 2)]
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[c.run(stream=s) for c, s in zip(cases, streams)] for _ in range(30)]
    torch.cuda.synchronize()
    for pair in got:
        for r, w in zip(pair, want):
            assert torch.equal(r.out, w.out) and torch.equal(r.lse, w.lse)


# ------------------------------------------------------- the step as a whole

def _step(c, state, new_kv, api, out):
    p = api.paged_plan(state["seq"], state["new"], state["held"], state["table"], state["free"], state["count"],
                       page_size=c.page, max_tokens=c.T, out=out["plan"])
    api.paged_append(new_kv[0], new_kv[1], p.slot_map, c.k_cache, c.v_cache)
    return p, api.paged_attention(c.q, c.k_cache, c.v_cache, state["table"], p.cu_new, p.kv_len, scale=c.scale,
                                  want_lse=True, out=out["attention"])


@pytest.mark.parametrize("captured", [False, True])
def test_plan_append_attend_in_stream_order(captured):
    """Each call reads what the one before it wrote, launched early or
    replayed from a graph, with the counts updated in place."""
    import torch
    from speculative_decoding_verification_25_gb300 import api
    c = PagedCase([(37, 5), (160, 5), (5, 5)], 8, 2, 64, 16, "bf16", seed=4)
    dev = "cuda:0"
    # before the step the last five tokens are not in the cache, nor their pages in the table
    new = torch.cat([torch.from_numpy(kv[:, -5:]).to(torch.bfloat16) for kv in c.host], 1).to(dev)
    old = [L - 5 for L, _ in c.rows]
    held = [-(-L // 16) for L in old]
    free = [int(c.block_table[b, p]) for b, (L, _) in enumerate(c.rows) for p in range(held[b], -(-L // 16))]
    fresh = dict(seq=_device(old), new=_device([5, 5, 5]), held=_device(held), table=c.block_table.clone(),
                 free=_device(free[::-1] + [0] * (c.k_cache.shape[0] - len(free))), count=_device([len(free)]))
    for b, (L, _) in enumerate(c.rows):
        fresh["table"][b, held[b]:] = 2 ** 31 - 1
        for at in range(old[b], L):
            c.k_cache[c.block_table[b, at // 16], :, at % 16] = float("nan")
            c.v_cache[c.block_table[b, at // 16], :, at % 16] = float("nan")
    state = {k: v.clone() for k, v in fresh.items()}
    e = lambda *n, d=torch.int32: torch.empty(*n, dtype=d, device=dev)
    out = dict(plan=api.PagedPlan(e(4), e(3), e(c.T), e(c.T), state["held"], state["count"]),
               attention=api.AttentionResult(e(c.T, 8, 64, d=torch.bfloat16), e(c.T, 8, d=torch.float32)))
    if captured:
        _step(c, state, new, api, out)   # the first call sets up the device and the workspace
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            api.attention_workspace(64, torch.device(dev))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            _step(c, state, new, api, out)
    for _ in range(3):
        for k in state:
            state[k].copy_(fresh[k])
        if captured:
            graph.replay()
        else:
            _step(c, state, new, api, out)
        torch.cuda.synchronize()
        assert out["plan"].kv_len.tolist() == [L for L, _ in c.rows] and state["count"].tolist() == [0]
        c.check(out["attention"])
