"""Every variant of the attention over the 4-bit cache by its type, head dimension
and form; captured calls; waits that run out; the checked build; and the operators
together, as a step uses them."""
from __future__ import annotations

import contextlib

import numpy as np
import pytest

import test_gpu_fp4 as attention
import test_gpu_rotary as rotary
from fp4_util import Fp4Case
from oracle import paged_fp4 as oracle
from test_gpu_paged import _holes, _rows

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def library():
    import torch
    from speculative_decoding_verification_25_gb300 import build as b
    b.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _form(c):
    """The host's choice, by the mean of a request's query rows of a key head."""
    G, rows, n = c.Hq // c.Hk, c.T * (c.Hq // c.Hk), max(1, len(c.rows))
    return "wide" if rows > 128 * n else "narrow" if G > 32 or rows > 32 * n else "32" if G > 16 or rows > 16 * n else "16"


# rows, Hq, Hk, page
SHAPES = {
    "16": {
        "tokens": (_rows(31, 50, 2600, 1), 32, 8, 16),
        "mixed": (_holes(_rows(32, 60, 1900, 6)), 12, 4, 32),       # requests of more than a unit among them
        "edges": ([(L, min(L, 3)) for L in (1, 2, 7, 8, 9, 31, 32, 33, 63, 65, 126, 127, 128, 129, 130, 255, 257)], 6, 2, 8),
        "split": ([(15013, 2), (70, 1)], 8, 1, 64),
    },
    "32": {
        "drafts": (_rows(41, 40, 2200, 9), 32, 8, 16),
        "group": (_rows(42, 30, 900, 1), 56, 2, 32),
        "edges": ([(L, min(L, 5)) for L in (1, 2, 7, 8, 9, 31, 33, 64, 127, 128, 129, 130, 255, 257)], 15, 3, 8),
        "split": ([(15013, 4), (70, 3)], 8, 1, 128),
    },
    "narrow": {
        "drafts": (_holes(_rows(33, 60, 1900, 17)), 24, 4, 32),
        "edges": ([(L, min(L, 20)) for L in (20, 127, 128, 129, 130, 131, 255, 256, 257, 385)], 12, 2, 8),
        "long": ([(15013, 12), (70, 9)], 8, 1, 64),
    },
    "wide": {
        "requests": (_rows(33, 40, 1500, 80), 16, 4, 32),
        "ragged": (_holes(_rows(34, 37, 1200, 167)), 14, 2, 8),
        "edges": ([(L, min(L, 70)) for L in (70, 127, 128, 129, 130, 255, 256, 257, 258, 300, 385)], 12, 3, 16),
        "prompt": ([(1111, 1111), (130, 130)], 4, 2, 256),
        "split": ([(7003, 200)], 6, 1, 64),
    },
}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("form,shape", [(f, s) for f in SHAPES for s in SHAPES[f]])
def test_every_variant(form, shape, D, dtype):
    rows, Hq, Hk, page = SHAPES[form][shape]
    c = Fp4Case(rows, Hq, Hk, D, page, dtype, seed=len(shape) + D, extra_tokens=len(shape) % 2)
    assert _form(c) == form
    c.check(c.run())


@pytest.mark.parametrize("form,shape", [(f, s) for f in SHAPES for s in SHAPES[f]])
def test_queries_of_any_size(form, shape):
    """Each unit or tile scales its bfloat16 queries by a power of two."""
    rows, Hq, Hk, page = SHAPES[form][shape]
    c = Fp4Case(rows[:12], Hq, Hk, 64, page, "bf16", seed=3)
    c.qkv.mul_(2.0 ** 70)
    c.qkv[1::3] *= 2.0 ** -24
    c.qkv[5::7] = 0
    c.scale = float(np.float32(c.scale * 2.0 ** -70))
    c.check(c.run())


def _same(got, want):
    import torch
    return torch.equal(got.out.view(torch.int16), want.out.view(torch.int16)) and torch.equal(got.lse, want.lse)


# ------------------------------------------------------------------ in graphs

@pytest.mark.parametrize("form", SHAPES)
def test_captured_without_a_workspace(form):
    """Two graphs captured cold on one stream, replayed in either order."""
    import torch
    rows, Hq, Hk, page = SHAPES[form]["edges"]
    c = Fp4Case(rows, Hq, Hk, 128, page, "bf16", seed=2)
    want = c.run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            graphs.append((graph, c.run()))
    for graph, got in (graphs[1], graphs[0], graphs[1]):
        got.out.fill_(float("nan"))
        got.lse.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert _same(got, want)


def test_both_caches_share_a_workspace():
    """Calls over 16-bit and 4-bit caches follow one another on a stream's workspace."""
    import torch
    from paged_util import PagedCase
    four = Fp4Case([(5000, 1), (100, 40), (3000, 3)], 8, 2, 128, 16, "bf16", seed=1)
    sixteen = PagedCase([(5000, 1), (100, 40), (3000, 3)], 8, 2, 128, 16, "bf16", seed=1)
    want = four.run(), sixteen.run()
    got = [(four.run(), sixteen.run()) for _ in range(10)]
    torch.cuda.synchronize()
    assert all(_same(g[0], want[0]) and _same(g[1], want[1]) for g in got)


# ---------------------------------------------------------- waits that run out

@pytest.fixture
def polls(monkeypatch):
    """Sets the limit of the checked library, which the Python calls use meanwhile."""
    from speculative_decoding_verification_25_gb300 import _native as N
    lib = N.load_checked()
    monkeypatch.setattr(N, "_lib", lib)
    yield lib.spec_checked_wait_polls_fp4
    lib.spec_checked_wait_polls_fp4(-1)


def _workspace(D):
    import torch
    from speculative_decoding_verification_25_gb300 import _native as N
    return torch.zeros(N.spec_paged_attention_workspace_bytes(D), dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("limit", [0, 1, 8, 16, 64])
@pytest.mark.parametrize("form,shape", [(f, s) for f in SHAPES for s in list(SHAPES[f])[::2]])
def test_waits_run_out(polls, form, shape, limit):
    """Wherever a call is given up: flagged, or right; the next one is right."""
    import torch
    from speculative_decoding_verification_25_gb300 import _native as N
    rows, Hq, Hk, page = SHAPES[form][shape]
    c = Fp4Case(rows, Hq, Hk, 128, page, "bf16", seed=8)
    want = c.run(workspace=_workspace(c.D))
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    polls(limit)
    for _ in range(4):
        flags.zero_()
        r = c.run(workspace=_workspace(c.D), flags=flags)
        assert flags.item() == N.SV_DEV_TIMEOUT or (flags.item() == 0 and _same(r, want))
        assert limit > 0 or flags.item() == N.SV_DEV_TIMEOUT
    polls(-1)
    flags.zero_()
    assert _same(c.run(workspace=_workspace(c.D), flags=flags), want) and flags.item() == 0


@pytest.mark.parametrize("form", SHAPES)
def test_a_call_that_gave_up_is_not_forgotten(polls, form):
    import torch
    from speculative_decoding_verification_25_gb300 import _native as N, api
    rows, Hq, Hk, page = SHAPES[form]["edges"]
    c = Fp4Case(rows, Hq, Hk, 64, page, "f16", seed=9, extra_tokens=2)
    ws = _workspace(64)
    want = c.run(workspace=ws)
    polls(0)
    c.run(workspace=ws)
    polls(-1)
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    r = c.run(workspace=ws, flags=flags)
    assert bool(r.out.isnan().all()) and bool(r.lse.isnan().all()) and flags.item() == N.SV_DEV_TIMEOUT
    assert api.attention_errors(ws) == N.SV_DEV_TIMEOUT and api.attention_errors(ws) == 0
    flags.zero_()
    assert _same(c.run(workspace=ws, flags=flags), want) and flags.item() == 0


# ------------------------------------------------------------- the checked build

@pytest.fixture
def checked(monkeypatch):
    from speculative_decoding_verification_25_gb300 import _native as N
    monkeypatch.setattr(N, "_lib", N.load_checked())


@pytest.mark.parametrize("name", list(attention.CASES)[::3])
def test_checked_attention(checked, name):
    import torch
    rows, *shape = attention.CASES[name]
    c = Fp4Case(rows, *shape, seed=len(name) + 1, extra_tokens=len(name) % 3)
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    c.check(c.run(flags=flags))
    assert flags.item() == 0


def test_checked_attention_of_bad_lengths_and_pages(checked):
    attention.test_attention_flags_bad_lengths_and_pages()
    attention.test_attention_of_no_requests()


@pytest.mark.parametrize("shape", rotary.SHAPES)
def test_checked_appends(checked, shape):
    rotary.test_append_rotary(shape)                 # no flag at all
    rotary.test_append_fp4_is_exact(shape, (0.25, 0.3))
    rotary.test_positions_and_slots_that_are_none()


# ------------------------------------------------------------------- together

def _ints(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("gains", [(1.0, 1.0), (0.5, 0.125)])
def test_plan_append_attend_in_stream_order(captured, gains):
    """A step over the 4-bit cache: the plan's positions and slots go to the rotated
    append, padding included, and the attention reads what it wrote."""
    import torch
    from speculative_decoding_verification_25_gb300 import api
    Hq, Hk, D, page, n, pad = 8, 2, 128, 16, 5, 3
    old = [37, 0, 160, 90]
    B, T = len(old), n * len(old) + pad
    g = torch.Generator().manual_seed(4)
    table = api.rotary_table(400, D, device=DEV)
    width = 12
    blocks = torch.randperm(60, generator=g).to(torch.int32)
    held = [-(-L // page) for L in old]
    cache = api.paged_cache_fp4(60, Hk, page, D, DEV)
    tables, at = torch.zeros(B, width, dtype=torch.int32), 0
    for b in range(B):
        tables[b, :held[b]] = blocks[at:at + held[b]]
        at += held[b]
    free = torch.cat([blocks[at:], torch.zeros(at, dtype=torch.int32)])
    qkv = torch.randn(T, Hq + 2 * Hk, D, generator=g).bfloat16().to(DEV)
    fresh = dict(seq=_ints(old), new=_ints([n] * B), held=_ints(held), table=tables.to(DEV), free=free.to(DEV),
                 count=_ints([60 - at]))
    # what is cached already goes through the same append, without a rotation
    past = torch.randn(sum(old), 2 * Hk, D, generator=g).bfloat16().to(DEV)
    slots = [int(tables[b, i // page]) * page + i % page for b in range(B) for i in range(old[b])]
    api.paged_append_fp4(None, past[:, :Hk], past[:, Hk:], None, None, _ints(slots), cache, k_gain=gains[0], v_gain=gains[1])
    state = {k: v.clone() for k, v in fresh.items()}
    e = lambda *s, d=torch.int32: torch.empty(*s, dtype=d, device=DEV)
    plan = api.PagedPlan(e(B + 1), e(B), e(T), e(T), state["held"], state["count"])
    result = api.AttentionResult(e(T, Hq, D, d=torch.bfloat16), e(T, Hq, d=torch.float32))
    q_out = e(T, Hq, D, d=torch.bfloat16)

    def step():
        p = api.paged_plan(state["seq"], state["new"], state["held"], state["table"], state["free"], state["count"],
                           page_size=page, max_tokens=T, out=plan)
        q = api.paged_append_fp4(qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], p.positions, table, p.slot_map, cache,
                                 k_gain=gains[0], v_gain=gains[1], q_out=q_out)
        api.paged_attention_fp4(q, cache, state["table"], p.cu_new, p.kv_len, k_gain=gains[0], v_gain=gains[1], out=result)

    if captured:
        step()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    for _ in range(3):
        for k in state:
            state[k].copy_(fresh[k])
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        assert plan.kv_len.tolist() == [L + n for L in old]
        turned = [oracle.rotate(x.double().cpu().numpy(), plan.positions.tolist(), table.double().cpu().numpy())
                  for x in (qkv[:, :Hq], qkv[:, Hq:Hq + Hk])]
        fresh_v = qkv[:, Hq + Hk:].double().cpu().numpy()
        out, lse = result.out.double().cpu().numpy(), result.lse.double().cpu().numpy()
        assert (out[n * B:] == 0).all() and np.isneginf(lse[n * B:]).all() and float(q_out[n * B:].abs().sum()) == 0
        q, first = q_out.double().cpu().numpy(), 0
        for b, L in enumerate(old):
            new = slice(b * n, (b + 1) * n)
            k, v = (np.concatenate([past[first:first + L, i * Hk:(i + 1) * Hk].double().cpu().numpy(), x[new]])
                    for i, x in ((0, turned[1]), (1, fresh_v)))
            k, v = (oracle.decode(*oracle.encode(x, gain), gain).transpose(1, 0, 2)[None] for x, gain in zip((k, v), gains))
            r = oracle.attention(q[new], k, v, [0, n], [L + n], D ** -0.5, "bf16")
            assert (np.abs(out[new] - r.out) <= r.out_tol).all() and (np.abs(lse[new] - r.lse) <= r.lse_tol).all()
            first += L


@pytest.mark.parametrize("start", [0, 4000])
def test_rotary_append_before_the_16_bit_attention(start):
    """The plan's positions to the rotated append, its cache and queries to paged_attention."""
    import torch
    from oracle import paged
    from speculative_decoding_verification_25_gb300 import api
    T, Hq, Hk, D, page = 40, 4, 2, 64, 8
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(T, Hq + 2 * Hk, D, generator=g).bfloat16().to(DEV)
    positions = torch.arange(start, start + T, dtype=torch.int32, device=DEV)
    table = api.rotary_table(5000, D, device=DEV)
    k, v = (torch.zeros(6, Hk, page, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q = api.paged_append_rotary(qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], positions, table,
                                torch.arange(T, dtype=torch.int32, device=DEV), k, v)
    got = api.paged_attention(q, k, v, _ints([list(range(6))]), _ints([0, T]), _ints([T]), want_lse=True)
    host = lambda x: x.double().cpu().numpy()
    want = oracle.rotate(host(qkv[:, :Hq]), positions.tolist(), host(table))
    tol = oracle.rotation_tolerance(host(qkv[:, :Hq]), want, positions.tolist(), host(table), "bf16")
    assert (np.abs(host(q) - want) <= tol).all()
    r = paged.attention(host(q), host(k), host(v), np.arange(6)[None], [0, T], [T], D ** -0.5, "bf16")
    assert (np.abs(host(got.out) - r.out) <= r.out_tol).all() and (np.abs(host(got.lse) - r.lse) <= r.lse_tol).all()


def test_every_call_is_made_on_the_tensors_device(monkeypatch):
    import torch
    from speculative_decoding_verification_25_gb300 import _native as N, api
    inside, seen, guard = [], [], api._device

    @contextlib.contextmanager
    def device(dev):
        inside.append(dev)
        with guard(dev):
            yield
        inside.pop()

    def watched(name, fn):
        def call(*args):
            assert inside and inside[-1] == torch.device("cuda", 0), name
            seen.append(name)
            return fn(*args)
        return call

    monkeypatch.setattr(api, "_device", device)
    names = ["spec_paged_append_rotary_raw", "spec_paged_append_fp4_raw", "spec_paged_read_fp4_raw", "spec_paged_attention_fp4_raw"]
    for name in names:
        monkeypatch.setattr(N, name, watched(name, getattr(N, name)))
    c = rotary.Case(6, 2, 1, 64, 32, False, 8, "bf16")
    api.paged_append_rotary(c.q, c.k_new, c.v_new, c.positions, c.table, c.slots, *c.random_caches())
    cache = c.random_cache_fp4()
    api.paged_append_fp4(c.q, c.k_new, c.v_new, c.positions, c.table, c.slots, cache)
    api.paged_read_fp4(cache, c.slots)
    api.paged_attention_fp4(c.q, cache, _ints([[0, 1]]), _ints([0, 6]), _ints([9]))
    torch.cuda.synchronize()
    assert seen == names


@pytest.mark.parametrize("fp4", [False, True])
def test_appends_on_a_stream_of_their_own(fp4):
    import torch
    from speculative_decoding_verification_25_gb300 import api
    c = rotary.Case(300, 8, 2, 128, 128, False, 16, "bf16", seed=1)
    side = torch.cuda.Stream()
    cache, (k, v) = c.random_cache_fp4(), c.random_caches()
    torch.cuda.synchronize()
    if fp4:
        q = api.paged_append_fp4(c.q, c.k_new, c.v_new, c.positions, c.table, c.slots, cache, stream=side)
        api.paged_read_fp4(cache, c.slots, stream=side)
    else:
        q = api.paged_append_rotary(c.q, c.k_new, c.v_new, c.positions, c.table, c.slots, k, v, stream=side)
    side.synchronize()
    c.check_rotated(q, c.q)
