"""What the paged cache operators refuse, on the host: statuses come before
any launch, and the Python calls name the argument (no call here reaches a
GPU)."""
import math

import pytest

FAKE = 0x10000   # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def N():
    from speculative_decoding_verification_25_gb300 import build as b
    b.build()
    from speculative_decoding_verification_25_gb300 import _native
    _native.load()
    return _native


PLAN = dict(seq=FAKE, new=FAKE, held=FAKE, table=FAKE, stack=FAKE, count=FAKE, B=3, page=16, max_pages=10, n_pages=50,
            max_tokens=20, cu=FAKE, kv=FAKE, slots=FAKE, pos=FAKE, held_out=FAKE, count_out=FAKE, flags=None, stream=None)
APPEND = dict(k=FAKE, ks=256, v=FAKE, vs=256, slots=FAKE, dtype=1, T=4, Hk=2, D=128, page=16, n_pages=9, kc=FAKE, vc=FAKE,
              flags=None, stream=None)
ATTEND = dict(q=FAKE, qs=1024, kc=FAKE, vc=FAKE, dtype=1, table=FAKE, cu=FAKE, kv=FAKE, B=2, T=4, Hq=8, Hk=2, D=128, page=16,
              max_pages=9, n_pages=50, scale=0.1, out=FAKE, lse=None, ws=FAKE, wsb=1 << 40, flags=None, stream=None)


def _plan(N, **kw):
    return N.spec_paged_plan_raw(*{**PLAN, **kw}.values())


def _append(N, **kw):
    return N.spec_paged_append_raw(*{**APPEND, **kw}.values())


def _attend(N, **kw):
    return N.spec_paged_attention_raw(*{**ATTEND, **kw}.values())


@pytest.mark.parametrize("bad", [dict(B=-1), dict(B=8193), dict(page=0), dict(page=4), dict(page=24), dict(page=512),
                                 dict(max_pages=0), dict(n_pages=0), dict(max_tokens=-1), dict(max_pages=1 << 27),
                                 dict(n_pages=1 << 27), dict(B=8192, max_pages=1 << 18)])
def test_plan_refuses_shapes(N, bad):
    assert _plan(N, **bad) == N.SV_ERR_SHAPE


def test_plan_refuses_pointers(N):
    for f in ("seq", "new", "held", "table", "stack", "count", "cu", "kv", "slots", "pos", "held_out", "count_out"):
        assert _plan(N, **{f: None}) == N.SV_ERR_NULL, f
        assert _plan(N, **{f: FAKE + 2}) == N.SV_ERR_ALIGN, f
    assert _plan(N, flags=FAKE + 1) == N.SV_ERR_ALIGN


@pytest.mark.parametrize("bad", [dict(T=-1), dict(Hk=0), dict(D=96), dict(D=0), dict(page=12), dict(n_pages=0),
                                 dict(n_pages=1 << 27), dict(ks=248), dict(vs=0)])
def test_append_refuses_shapes(N, bad):
    assert _append(N, **bad) == N.SV_ERR_SHAPE


def test_append_refuses_types_and_pointers(N):
    assert _append(N, dtype=N.SV_F32) == N.SV_ERR_DTYPE and _append(N, dtype=3) == N.SV_ERR_DTYPE
    for f in ("k", "v", "slots", "kc", "vc"):
        assert _append(N, **{f: None}) == N.SV_ERR_NULL, f
    for f in ("k", "v", "kc", "vc"):
        assert _append(N, **{f: FAKE + 8}) == N.SV_ERR_ALIGN, f
    assert _append(N, ks=260) == N.SV_ERR_ALIGN and _append(N, vs=257) == N.SV_ERR_ALIGN
    assert _append(N, slots=FAKE + 2) == N.SV_ERR_ALIGN and _append(N, flags=FAKE + 2) == N.SV_ERR_ALIGN
    assert _append(N, T=0, k=None, v=None, slots=None, kc=None, vc=None) == N.SV_OK


@pytest.mark.parametrize("bad", [dict(B=-1), dict(T=-1), dict(Hk=0), dict(Hq=7), dict(Hq=0), dict(Hq=258, qs=1 << 20),
                                 dict(D=80), dict(page=1), dict(max_pages=0), dict(n_pages=0), dict(n_pages=1 << 27),
                                 dict(max_pages=1 << 27), dict(qs=1016), dict(scale=0.0), dict(scale=-1.0),
                                 dict(scale=math.inf), dict(scale=math.nan)])
def test_attention_refuses_shapes(N, bad):
    assert _attend(N, **bad) == N.SV_ERR_SHAPE


def test_attention_refuses_types_pointers_and_workspaces(N):
    assert _attend(N, dtype=N.SV_F32) == N.SV_ERR_DTYPE and _attend(N, dtype=-1) == N.SV_ERR_DTYPE
    for f in ("q", "kc", "vc", "table", "cu", "kv", "out", "ws"):
        assert _attend(N, **{f: None}) == N.SV_ERR_NULL, f
    for f in ("q", "kc", "vc", "out", "ws"):
        assert _attend(N, **{f: FAKE + 8}) == N.SV_ERR_ALIGN, f
    for f in ("table", "cu", "kv", "lse", "flags"):
        assert _attend(N, **{f: FAKE + 2}) == N.SV_ERR_ALIGN, f
    assert _attend(N, qs=1028) == N.SV_ERR_ALIGN
    for D in (64, 128):
        need = N.spec_paged_attention_workspace_bytes(D)
        assert need >= N.SV_ATTENTION_COUNTER_BYTES
        assert _attend(N, D=D, wsb=need - 1) == N.SV_ERR_WORKSPACE
    assert N.spec_paged_attention_workspace_bytes(96) == 0
    assert _attend(N, T=0, q=None, out=None, ws=None, wsb=0) == N.SV_OK


def test_python_calls_refuse_host_tensors(N):
    import torch
    from speculative_decoding_verification_25_gb300 import api
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError, match="seq_len"):
        api.paged_plan(i(2), i(2), i(2), i(2, 3), i(9), i(1), page_size=16, max_tokens=4)
    k = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k_cache"):
        api.paged_append(k[:2, :, 0], k[:2, :, 0], i(2), k, k)
    with pytest.raises(ValueError, match="k_cache"):
        api.paged_attention(k[:2, :, 0], k, k, i(1, 3), i(2), i(1))
    with pytest.raises(TypeError, match="k_cache"):
        api.paged_attention(k[:2, :, 0], k.float(), k, i(1, 3), i(2), i(1))
