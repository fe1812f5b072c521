"""The Python calls launch on their tensors' device, whichever one is current,
and refuse streams of another device."""
from __future__ import annotations

import contextlib

import pytest
import torch


@pytest.fixture
def api():
    from speculative_decoding_verification_25_gb300 import build as b
    b.build()
    from speculative_decoding_verification_25_gb300 import api
    return api


class FakeStream:
    def __init__(self, index):
        self.device, self.cuda_stream = torch.device("cuda", index), 7


@pytest.mark.parametrize("current", [0, 1, 3])
def test_another_current_device_is_left_for_the_call(api, monkeypatch, current):
    entered = []

    @contextlib.contextmanager
    def device(dev):
        entered.append(dev)
        yield

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
    monkeypatch.setattr(torch.cuda, "device", device)
    with api._device(torch.device("cuda", 1)):
        pass
    assert entered == ([] if current == 1 else [torch.device("cuda", 1)])


def test_streams_of_another_device_are_refused(api):
    dev = torch.device("cuda", 1)
    mine = FakeStream(1)
    assert api._stream(mine, dev) is mine and api._stream_handle(mine, dev) == 7
    for call in (api._stream, api._stream_handle):
        with pytest.raises(ValueError, match="stream is on cuda:0, expected cuda:1"):
            call(FakeStream(0), dev)


@pytest.mark.gpu
def test_every_call_of_the_library_is_made_on_the_tensors_device(api, monkeypatch):
    """Each entry point that launches is called within the guard, for that device."""
    from speculative_decoding_verification_25_gb300 import _native as N
    from paged_util import PagedCase
    inside, seen = [], []
    guard = api._device

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
    for name in dir(N):
        if name.endswith("_raw") and name != "spec_verify_row_stats_raw" or name.endswith("device_errors"):
            monkeypatch.setattr(N, name, watched(name, getattr(N, name)))

    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda:0")
    B, K, V = 2, 3, 512
    logits = torch.randn(B, K + 1, V, device="cuda:0")
    args = (logits, logits[:, :K].contiguous(), i32(B, K), torch.rand(B, K + 1, device="cuda:0"),
            torch.ones(B, device="cuda:0"))
    result = api.spec_verify(*args)
    api.spec_verify(*args, k_per_row=i32(B))
    api.spec_verify_and_plug(*args, i32(B, 64), i32(B))
    api.plug(result, i32(B, 64), i32(B))
    api.verify_tree(logits, i32(B, K), i32(B, K) - 1)
    api.device_errors(api.workspace_for(B, K, V, N.SV_F32, torch.device("cuda:0")))
    api.paged_plan(i32(2), i32(2), i32(2), i32(2, 3), i32(9), i32(1), page_size=16, max_tokens=4)
    c = PagedCase([(40, 3)], 4, 2, 64, 16, "bf16")
    api.paged_append(c.qkv[:, 4:6], c.qkv[:, 6:], i32(3) - 1, c.k_cache, c.v_cache)
    c.run()
    api.attention_errors(api.attention_workspace(64, torch.device("cuda:0")))
    torch.cuda.synchronize()
    assert set(seen) == {"spec_verify_raw", "spec_verify_ragged_raw", "spec_verify_and_plug_raw", "spec_verify_plug_raw",
                         "spec_verify_tree_raw", "spec_verify_device_errors", "spec_paged_plan_raw",
                         "spec_paged_append_raw", "spec_paged_attention_raw", "spec_paged_attention_device_errors"}
