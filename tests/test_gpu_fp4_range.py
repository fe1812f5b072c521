"""Attention over the 4-bit cache at the ends of its arguments' ranges: gains, scales
and queries far from 1, rows whose probabilities differ by far, the longest context."""
from __future__ import annotations

import math

import numpy as np
import pytest

from fp4_util import Fp4Case
from oracle import paged as paged_oracle
from oracle import paged_fp4 as oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
# new tokens of a request that take each form, with groups of 4
FORMS = {"16": 3, "32": 7, "narrow": 20, "wide": 70}
PAGE = 256


@pytest.fixture(scope="module", autouse=True)
def library():
    import torch
    from speculative_decoding_verification_25_gb300 import build as b
    b.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _shared(k, v, q, B, repeat=1, gains=(1.0, 1.0), scale=1.0, cut=0):
    """B requests of the same queries [n, G, D] on one key head, whose cache is the pages
    of k and v [L, D] `repeat` times, without the last `cut` keys."""
    import torch
    from speculative_decoding_verification_25_gb300 import api
    (L, D), (n, G, _) = k.shape, q.shape
    pages = L // PAGE
    parts = []
    for x, gain in ((k, gains[0]), (v, gains[1])):
        codes, scales = oracle.encode(x.reshape(pages, 1, PAGE, D), gain)
        parts += [torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV).view(torch.float8_e4m3fn)]
    table = torch.arange(pages, dtype=torch.int32, device=DEV).repeat(B, repeat)
    length = torch.full((B,), L * repeat - cut, dtype=torch.int32, device=DEV)
    queries = torch.from_numpy(q).to(torch.bfloat16).to(DEV).repeat(B, 1, 1)
    cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device=DEV)
    return api.paged_attention_fp4(queries, api.PagedCacheFp4(*parts), table, cu, length, scale=scale, k_gain=gains[0],
                                   v_gain=gains[1], want_lse=True)


def _bf16(x):
    import torch
    return torch.from_numpy(np.asarray(x, np.float64)).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("cut", [0, 5])
@pytest.mark.parametrize("form", FORMS)
def test_attention_over_the_most_keys(form, cut):
    """2^31 - 1024 keys, the same pages over and over: each has its weight among the 1024."""
    n, G, D, L, repeat = FORMS[form], 4, 64, 4 * PAGE, 2 ** 21 - 1
    rng = np.random.default_rng(len(form))
    k, v = rng.normal(size=(2, L, D))
    q = _bf16(rng.normal(size=(n, G, D)) / 8)
    r = _shared(k, v, q, 1, repeat=repeat, cut=cut)
    k, v = (oracle.decode(*oracle.encode(x))[None, None] for x in (k, v))
    # every token sees all of a period: as if the queries stood behind them
    want = paged_oracle.attention(np.broadcast_to(q, (n, G, D)).reshape(1, n * G, D), k, v, np.zeros((1, 1), int), [0, 1], [L],
                                  1.0, "f16")
    out, lse = r.out.double().cpu().numpy().reshape(1, n * G, D), r.lse.double().cpu().numpy().reshape(1, n * G)
    # Float32 sums of up to 2^31 / 152 keys, 16 at a time, which may truncate, and of as many
    # parts as there are CTAs; up to n + cut of the 2^31 keys are not seen.  One rounding to bfloat16.
    adds = (2.0 ** 31 / 152 / 16 + 320) * 2.0 ** -23
    few = (n + cut) / 2.0 ** 31
    weights = np.exp(q.reshape(n * G, D) @ k[0, 0].T)
    spread = weights / weights.sum(-1, keepdims=True) @ np.abs(v[0, 0])
    tol = want.out_tol + 2 * (adds + few * L) * spread + 2.0 ** -8 * np.abs(want.out)
    assert (np.abs(out - want.out) <= tol).all()
    assert (np.abs(lse - want.lse - math.log(repeat)) <= want.lse_tol + adds + few * L + 2.0 ** -20).all()


@pytest.mark.parametrize("below", [6.0, 14.0, 16.0, 17.5])
@pytest.mark.parametrize("form", FORMS)
def test_a_key_that_outweighs_the_others(form, below):
    """The first key's score is `below` above all others', its value is 0: what remains
    are the others' small probabilities.  They are rounded to 11 bits, or where they are
    less than 2^-21 of the largest to steps of 2^-31 of it, so by half of that."""
    n, G, D, L, B = FORMS[form], 4, 64, 4096, 320
    k, v = np.zeros((L, D)), np.ones((L, D))
    k[0, 0], k[1:, 0], v[0] = 6, -6, 0
    q = np.zeros((n, G, D))
    q[..., 0] = _bf16(below / 12)
    r = _shared(k, v, q, B)
    out, lse = (x.double().cpu().numpy().reshape(B, n, G, -1) for x in (r.out, r.lse))
    k, v = (oracle.decode(*oracle.encode(x))[None, None] for x in (k, v))
    want = paged_oracle.attention(q, k, v, np.zeros((1, 1), int), [0, n], [L], 1.0, "f16")
    # the oracle's bound is for steps of 2^-24 of the largest
    others = np.abs(v).sum() / D
    tol = want.out_tol - 1.01 * (2.0 ** -25 - 2.0 ** -32) * others + 2.0 ** -8 * np.abs(want.out)
    assert (tol > 0).all() and (tol < 0.02 * np.abs(want.out)).all()
    assert (np.abs(out - want.out) <= tol).all()
    assert (np.abs(lse[..., 0] - want.lse) <= want.lse_tol).all()


@pytest.mark.parametrize("gain", [1e30, 1e-30])
@pytest.mark.parametrize("form", FORMS)
def test_parts_of_a_long_sum_with_an_extreme_gain(form, gain):
    """One request cut into parts of 200000 or more keys, all of the largest value: a part's
    sum times the gain is past float32's range, the results are not."""
    n, G, D = FORMS[form], 4, 64
    gain = float(np.float32(gain))
    L, repeat = 40 * PAGE, 6000           # 61 million keys
    v = np.full((L, D), 6 * 448 * gain)
    r = _shared(np.zeros((L, D)), v, np.ones((n, G, D)), 1, repeat=repeat, gains=(1.0, gain))
    # A sum of N float32 additions that may truncate is within N 2^-23: a range's products add
    # 16 keys at a time, the join a part at a time; the normaliser as much; one rounding.
    keys = L * repeat
    adds = keys / 152 / 16 + 320
    tol = 2 * adds * 2.0 ** -23 + 2.0 ** -8
    assert tol < 0.02
    assert bool(((r.out.double() / (2688 * gain) - 1).abs() <= tol).all())
    # tokens before the last see some keys less: at most n of 61 million
    assert bool(((r.lse.double() - math.log(keys)).abs() <= adds * 2.0 ** -23 + n / keys + 2.0 ** -20).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("form", FORMS)
def test_scores_too_small_for_float32(form, D):
    """scale * log2(e) * k_gain times the power of two of the queries underflows: every
    score is 0 to all purposes, and masked keys are masked all the same."""
    n = FORMS[form]
    c = Fp4Case([(300, n), (n + 133, n), (n, n)], 8, 2, D, 16, "bf16", seed=4, gains=(float(np.float32(1e-20)), 1.0))
    c.qkv.mul_(1e-24)
    c.check(c.run())


@pytest.mark.parametrize("form", FORMS)
def test_rows_of_zeros_beside_scores_past_float32(form):
    """Queries so large that the factor of their scores overflows: rows of zeros in the
    same unit have scores of 0."""
    n = FORMS[form]
    c = Fp4Case([(300, n), (n + 133, n)], 8, 2, 64, 16, "bf16", seed=4)
    c.scale = 1e30
    want = c.host[0][1][:300 - n + 1].mean(0)      # token 0 of the first request: a uniform average
    c.qkv.mul_(1e30)
    c.qkv[0, 0] = 0
    r = c.run()
    got = r.out[0, 0].double().cpu().numpy()
    # sums of values of up to 301 keys, P exact, one rounding each of P's inverse sum and of the result
    assert (np.abs(got - want[0]) <= 2.0 ** -8 * np.abs(want[0]) + 2.0 ** -20).all()
    assert abs(float(r.lse[0, 0]) - math.log(300 - n + 1)) <= 2.0 ** -20


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("form", FORMS)
def test_rows_that_differ_by_far_at_ordinary_sizes(form, D):
    """Queries of about 1 beside others 2^-20 of that in the same unit, whose scores matter
    since the keys are large."""
    n = FORMS[form]
    c = Fp4Case([(700, n), (n, n), (n + 250, n)], 8, 2, D, 16, "bf16", seed=21)
    c.qkv[::3, ::2] *= 2.0 ** -20
    c.qkv[1::3, 1::4] *= 2.0 ** -22
    c.k_cache.mul_(2.0 ** 20)
    for kv in c.host:
        kv[0] *= 2.0 ** 20
    c.gains = (2.0 ** 20, 1.0)
    c.encode()
    c.check(c.run())


@pytest.mark.parametrize("factor", [2.0 ** -50, 1.0, 2.0 ** 60])
@pytest.mark.parametrize("form", FORMS)
def test_queries_that_are_not_finite_beside_others(form, factor):
    """Rows of NaN and infinities leave the power of two of their unit to the others."""
    n = FORMS[form]
    c = Fp4Case([(300, n), (n + 133, n), (n, n)], 8, 2, 64, 16, "bf16", seed=9)
    c.qkv.mul_(factor)
    c.scale = float(np.float32(c.scale / factor))
    c.qkv[1::n, 2], c.qkv[2::n, 5, 7], c.qkv[0, 6, 60] = float("nan"), float("inf"), -float("inf")
    bad = ~c.q.isfinite().all(-1).cpu().numpy()
    r = c.run()
    out, lse = r.out.double().cpu().numpy(), r.lse.double().cpu().numpy()
    c.qkv.nan_to_num_(0.0, 0.0, 0.0)      # the oracle's rows are each by itself
    want = c.reference()
    assert bad.sum() == 7 and np.isnan(out[bad]).all() and np.isnan(lse[bad]).all()
    assert (np.abs(out - want.out) <= want.out_tol)[~bad].all() and (np.abs(lse - want.lse) <= want.lse_tol)[~bad].all()
