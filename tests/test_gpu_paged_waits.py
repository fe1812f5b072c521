"""A wait inside the attention kernel that runs out: the kernel says so, ends
with nothing of its own in flight, and the next call is right.  The checked
build takes a limit of polls; none at all ends every wait at once."""
from __future__ import annotations

import pytest

from paged_util import PagedCase
from test_gpu_paged import CASES

pytestmark = pytest.mark.gpu

NAMES = ["one_token", "verify", "long_draft", "prompt", "prompt_64", "many_tiles", "ragged_units", "split", "split_wide"]


@pytest.fixture
def polls(monkeypatch):
    """Sets the limit of the checked library, which the Python calls use meanwhile."""
    import torch
    from speculative_decoding_verification_25_gb300 import _native as N
    from speculative_decoding_verification_25_gb300 import build as b
    b.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    lib = N.load_checked()
    monkeypatch.setattr(N, "_lib", lib)
    yield lib.spec_checked_wait_polls
    lib.spec_checked_wait_polls(-1)


def _workspace(D):
    import torch
    from speculative_decoding_verification_25_gb300 import _native as N
    return torch.zeros(N.spec_paged_attention_workspace_bytes(D), dtype=torch.uint8, device="cuda:0")


def _same(r, want):
    import torch
    return torch.equal(r.out.view(torch.int16), want.out.view(torch.int16)) and torch.equal(r.lse, want.lse)


@pytest.mark.parametrize("name", NAMES)
def test_every_wait_ends_at_once(polls, name):
    import torch
    from speculative_decoding_verification_25_gb300 import _native as N
    rows, *shape = CASES[name]
    c = PagedCase(rows, *shape, seed=7)
    want = c.run(workspace=_workspace(c.D))
    c.check(want)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    polls(0)
    for _ in range(3):
        c.run(workspace=_workspace(c.D), flags=flags)
    torch.cuda.synchronize()
    assert flags.item() == N.SV_DEV_TIMEOUT
    polls(-1)
    flags.zero_()
    assert _same(c.run(workspace=_workspace(c.D), flags=flags), want) and flags.item() == 0


@pytest.mark.parametrize("limit", [1, 2, 4, 16])
@pytest.mark.parametrize("name", NAMES)
def test_some_waits_run_out(polls, name, limit):
    """Wherever the walk is given up: flagged, or right."""
    import torch
    from speculative_decoding_verification_25_gb300 import _native as N
    rows, *shape = CASES[name]
    c = PagedCase(rows, *shape, seed=8)
    want = c.run(workspace=_workspace(c.D))
    flags = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    polls(limit)
    for _ in range(5):
        flags.zero_()
        r = c.run(workspace=_workspace(c.D), flags=flags)
        assert flags.item() == N.SV_DEV_TIMEOUT or (flags.item() == 0 and _same(r, want))
    polls(-1)
    flags.zero_()
    assert _same(c.run(workspace=_workspace(c.D), flags=flags), want) and flags.item() == 0


@pytest.mark.parametrize("name", ["verify", "prompt", "split", "split_wide"])
def test_a_call_that_gave_up_is_not_forgotten(polls, name):
    """Calls on the same workspace give NaN and the flag until it is cleared,
    whoever asks: flags are optional, the workspace remembers."""
    import torch
    from speculative_decoding_verification_25_gb300 import _native as N, api
    rows, *shape = CASES[name]
    c = PagedCase(rows, *shape, seed=9, extra_tokens=2)
    want = c.run()
    ws = api.attention_workspace(c.D, torch.device("cuda:0"))
    assert api.attention_errors(ws) == 0
    polls(0)
    c.run()
    polls(-1)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    for _ in range(2):
        r = c.run(flags=flags)
        assert bool(r.out.isnan().all()) and bool(r.lse.isnan().all()) and flags.item() == N.SV_DEV_TIMEOUT
    assert api.attention_errors(ws) == N.SV_DEV_TIMEOUT
    assert api.attention_errors(ws) == 0 and int(ws[:N.SV_ATTENTION_COUNTER_BYTES].sum()) == 0
    flags.zero_()
    assert _same(c.run(flags=flags), want) and flags.item() == 0
    assert api.attention_errors(ws) == 0
