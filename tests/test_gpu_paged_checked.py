"""The paged operators in the checked build (libspec_verify_checked.so): every
global index that their kernels form is tested against its array.  No call may
raise SV_DEV_OUT_OF_BOUNDS, and results must still match the oracle."""
from __future__ import annotations

import numpy as np
import pytest

import test_gpu_paged as plain
from oracle import paged as oracle
from paged_util import PagedCase

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def checked(monkeypatch):
    """The Python calls use the checked library."""
    import torch
    from speculative_decoding_verification_25_gb300 import _native as N
    from speculative_decoding_verification_25_gb300 import build as b
    b.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    monkeypatch.setattr(N, "_lib", N.load_checked())


@pytest.mark.parametrize("B,page,width,n_max", [(1, 16, 9, 5), (2, 8, 3, 1), (31, 8, 40, 17), (300, 256, 5, 700),
                                                (1025, 8, 9, 20), (8192, 8, 4, 2), (3, 128, 600, 60000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(B, page, width, n_max, in_place):
    plain.test_plan_matches_the_oracle(B, page, width, n_max, in_place)   # no flag at all


@pytest.mark.parametrize("B,page,width,n_max", [(7, 8, 5, 9), (64, 16, 20, 33), (1500, 8, 8, 11)])
@pytest.mark.parametrize("short", ["pages", "tokens", "both", "none"])
def test_plan_of_rows_that_cannot_be_served(B, page, width, n_max, short):
    from speculative_decoding_verification_25_gb300 import _native as N
    rng = np.random.default_rng(B * len(short))
    seq, new, held, table, stack, n_pages = plain._plan_state(rng, B, page, width, n_max, broken=True)
    ok = (seq >= 0) & (new >= 0)
    max_tokens = int(new[ok].sum()) // (2 if short in ("tokens", "both") else 1) + 1
    if short in ("pages", "both"):
        stack = stack[:len(stack) // 5]
    ref = oracle.plan(seq, new, held, table.astype(np.int32), stack, page, max_tokens)
    got, t, flags = plain._run_plan(seq, new, held, table, stack, n_pages, page, max_tokens)
    plain._compare_plan(got, t, ref)
    assert not flags & N.SV_DEV_OUT_OF_BOUNDS


def test_plan_of_no_rows_and_of_bad_pages():
    plain.test_plan_of_no_rows_and_of_no_tokens()
    plain.test_plan_flags_pages_outside_the_cache()


@pytest.mark.parametrize("T,Hk,D,page,dtype", [(1, 1, 64, 8, "bf16"), (333, 3, 64, 32, "f16"), (2049, 8, 128, 256, "f16")])
def test_append(T, Hk, D, page, dtype):
    plain.test_append_is_bit_exact(T, Hk, D, page, dtype)
    plain.test_append_skips_slots_past_the_cache()


@pytest.mark.parametrize("name", plain.CASES)
def test_attention(name):
    import torch
    rows, *shape = plain.CASES[name]
    c = PagedCase(rows, *shape, seed=len(name) + 1, extra_tokens=len(name) % 3)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    c.check(c.run(flags=flags))
    assert flags.item() == 0


def test_attention_of_bad_lengths_and_pages():
    plain.test_attention_flags_bad_lengths_and_pages()
    plain.test_attention_of_no_requests()
