"""What the rotated appends and the 4-bit cache's operators refuse on the host:
statuses come before any launch, and the Python calls name the argument (no call
here reaches a GPU)."""
import math

import pytest
import torch

from test_paged_refusals import FakeCuda

FAKE = 0x10000   # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def N():
    from speculative_decoding_verification_25_gb300 import build as b
    b.build()
    from speculative_decoding_verification_25_gb300 import _native
    _native.load()
    return _native


COMMON = dict(q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, pos=FAKE, table=FAKE, most=100, rot=128, inter=0, slots=FAKE,
              dtype=1, T=4, Hq=8, Hk=2, D=128, page=16, n_pages=9)
ROTARY = dict(COMMON, out=FAKE, outs=1024, kc=FAKE, vc=FAKE, flags=None, stream=None)
FP4 = dict(COMMON, kg=1.0, vg=1.0, out=FAKE, outs=1024, kc=FAKE, ksc=FAKE, vc=FAKE, vsc=FAKE, flags=None, stream=None)
READ = dict(kc=FAKE, ksc=FAKE, vc=FAKE, vsc=FAKE, slots=FAKE, dtype=1, T=4, Hk=2, D=128, page=16, n_pages=9, kg=1.0, vg=1.0,
            k=FAKE, v=FAKE, flags=None, stream=None)
ATTEND = dict(q=FAKE, qs=1024, kc=FAKE, ksc=FAKE, vc=FAKE, vsc=FAKE, dtype=1, table=FAKE, cu=FAKE, kv=FAKE, B=2, T=4, Hq=8,
              Hk=2, D=128, page=16, max_pages=9, n_pages=50, scale=0.1, kg=1.0, vg=1.0, out=FAKE, lse=None, ws=FAKE,
              wsb=1 << 40, flags=None, stream=None)


def _rotary(N, **kw):
    return N.spec_paged_append_rotary_raw(*{**ROTARY, **kw}.values())


def _fp4(N, **kw):
    return N.spec_paged_append_fp4_raw(*{**FP4, **kw}.values())


def _read(N, **kw):
    return N.spec_paged_read_fp4_raw(*{**READ, **kw}.values())


def _attend(N, **kw):
    return N.spec_paged_attention_fp4_raw(*{**ATTEND, **kw}.values())


GAINS = [dict(kg=0.0), dict(vg=-1.0), dict(kg=math.nan), dict(vg=math.inf), dict(kg=1e-31), dict(vg=1e31)]


@pytest.mark.parametrize("bad", [dict(T=-1), dict(Hk=0), dict(Hk=5000), dict(Hq=-1), dict(Hq=5000, qs=1 << 20, outs=1 << 20),
                                 dict(D=96), dict(page=12), dict(n_pages=0), dict(n_pages=1 << 27), dict(ks=248), dict(vs=0),
                                 dict(qs=1016), dict(outs=0), dict(most=0), dict(rot=0), dict(rot=16), dict(rot=48),
                                 dict(rot=160), dict(D=64, rot=96)])
def test_appends_refuse_shapes(N, bad):
    assert _rotary(N, **bad) == N.SV_ERR_SHAPE
    assert _fp4(N, **bad) == N.SV_ERR_SHAPE


@pytest.mark.parametrize("bad", GAINS)
def test_gains_are_positive_and_far_from_the_ends_of_float32(N, bad):
    assert _fp4(N, **bad) == N.SV_ERR_SHAPE and _read(N, **bad) == N.SV_ERR_SHAPE and _attend(N, **bad) == N.SV_ERR_SHAPE


def test_appends_refuse_types_and_pointers(N):
    for call, arrays in ((_rotary, ("kc", "vc")), (_fp4, ("kc", "ksc", "vc", "vsc"))):
        assert call(N, dtype=N.SV_F32) == N.SV_ERR_DTYPE
        for f in ("q", "k", "v", "slots", "out") + arrays:
            assert call(N, **{f: None}) == N.SV_ERR_NULL, f
        for f in ("q", "k", "v", "table", "out", "kc", "vc"):
            assert call(N, **{f: FAKE + 8}) == N.SV_ERR_ALIGN, f
        for f in ("slots", "pos", "flags"):
            assert call(N, **{f: FAKE + 2}) == N.SV_ERR_ALIGN, f
        for f in ("qs", "ks", "vs", "outs"):
            assert call(N, **{f: 1028}) == N.SV_ERR_ALIGN, f
        assert call(N, T=0, q=None, k=None, v=None, slots=None, out=None) == N.SV_OK
    # without positions there is no rotation, and queries have nothing to wait for
    assert _rotary(N, pos=None, table=None) == N.SV_ERR_NULL and _rotary(N, table=None) == N.SV_ERR_NULL
    assert _fp4(N, pos=None, table=None) == N.SV_ERR_SHAPE
    assert _fp4(N, pos=None) == N.SV_ERR_NULL and _fp4(N, table=None) == N.SV_ERR_NULL
    assert _fp4(N, pos=None, table=None, Hq=0, k=None) == N.SV_ERR_NULL   # the shape passes


@pytest.mark.parametrize("bad", [dict(T=-1), dict(Hk=0), dict(D=32), dict(page=7), dict(n_pages=0), dict(n_pages=1 << 27),
                                 dict(T=2 ** 31 - 1, Hk=4096)])
def test_read_refuses_shapes(N, bad):
    assert _read(N, **bad) == N.SV_ERR_SHAPE


def test_read_refuses_types_and_pointers(N):
    assert _read(N, dtype=N.SV_F32) == N.SV_ERR_DTYPE
    for f in ("kc", "ksc", "vc", "vsc", "slots", "k", "v"):
        assert _read(N, **{f: None}) == N.SV_ERR_NULL, f
    for f in ("kc", "vc", "k", "v"):
        assert _read(N, **{f: FAKE + 8}) == N.SV_ERR_ALIGN, f
    assert _read(N, slots=FAKE + 2) == N.SV_ERR_ALIGN and _read(N, T=0, k=None) == N.SV_OK


@pytest.mark.parametrize("bad", [dict(B=-1), dict(T=-1), dict(Hk=0), dict(Hq=7), dict(Hq=0), dict(Hq=258, qs=1 << 20),
                                 dict(D=80), dict(page=1), dict(max_pages=0), dict(n_pages=0), dict(n_pages=1 << 27),
                                 dict(max_pages=1 << 27), dict(qs=1016), dict(scale=0.0), dict(scale=-1.0),
                                 dict(scale=math.inf), dict(scale=math.nan), dict(scale=3e38), dict(scale=1e-20, kg=1e-20),
                                 dict(scale=1e20, kg=1e20), dict(page=16, max_pages=(2 ** 31 - 512) // 16 + 1)])
def test_attention_refuses_shapes(N, bad):
    assert _attend(N, **bad) == N.SV_ERR_SHAPE


def test_attention_refuses_types_pointers_and_workspaces(N):
    assert _attend(N, dtype=N.SV_F32) == N.SV_ERR_DTYPE and _attend(N, dtype=-1) == N.SV_ERR_DTYPE
    for f in ("q", "kc", "ksc", "vc", "vsc", "table", "cu", "kv", "out", "ws"):
        assert _attend(N, **{f: None}) == N.SV_ERR_NULL, f
    for f in ("q", "kc", "ksc", "vc", "vsc", "out", "ws"):
        assert _attend(N, **{f: FAKE + 8}) == N.SV_ERR_ALIGN, f
    for f in ("table", "cu", "kv", "lse", "flags"):
        assert _attend(N, **{f: FAKE + 2}) == N.SV_ERR_ALIGN, f
    assert _attend(N, qs=1028) == N.SV_ERR_ALIGN
    for D in (64, 128):
        assert _attend(N, D=D, wsb=N.spec_paged_attention_workspace_bytes(D) - 1) == N.SV_ERR_WORKSPACE
    assert _attend(N, T=0, q=None, out=None, ws=None, wsb=0) == N.SV_OK


def test_python_calls_name_the_argument(N):
    from speculative_decoding_verification_25_gb300 import api
    cuda = lambda t: t.as_subclass(FakeCuda)
    i = lambda *s: cuda(torch.zeros(*s, dtype=torch.int32))
    b = lambda *s: cuda(torch.zeros(*s, dtype=torch.bfloat16))
    kv, table = b(3, 2, 16, 64), cuda(torch.zeros(50, 64))
    with pytest.raises(ValueError, match="invalid head dimension"):
        api.paged_cache_fp4(3, 2, 16, 96)
    good = api.PagedCacheFp4(*[cuda(t) for t in api.paged_cache_fp4(3, 2, 16, 64)])
    host = api.paged_cache_fp4(3, 2, 16, 64)
    assert host.k.shape == (3, 2, 16, 32) and host.v_scale.shape == (3, 2, 16, 4)
    for call in (lambda c: api.paged_append_fp4(None, b(4, 2, 64), b(4, 2, 64), None, None, i(4), c),
                 lambda c: api.paged_read_fp4(c, i(4)),
                 lambda c: api.paged_attention_fp4(b(4, 4, 64), c, i(2, 3), i(3), i(2))):
        with pytest.raises(ValueError, match="cache.k must be a CUDA tensor"):
            call(host)
        with pytest.raises(TypeError, match="cache.k_scale"):
            call(good._replace(k_scale=cuda(good.k_scale.view(torch.uint8))))
        with pytest.raises(ValueError, match="cache.v must have shape"):
            call(good._replace(v=cuda(torch.zeros(3, 2, 16, 64, dtype=torch.uint8))))
        with pytest.raises(ValueError, match="cache.k must be"):
            call(good._replace(k=cuda(torch.zeros(3, 2, 16, dtype=torch.uint8))))
    with pytest.raises(ValueError, match="come together"):
        api.paged_append_fp4(None, b(4, 2, 64), b(4, 2, 64), i(4), None, i(4), good)
    with pytest.raises(ValueError, match="q needs positions"):
        api.paged_append_fp4(b(4, 4, 64), b(4, 2, 64), b(4, 2, 64), None, None, i(4), good)
    with pytest.raises(TypeError, match="k_new dtype"):
        api.paged_append_fp4(None, cuda(torch.zeros(4, 2, 64)), b(4, 2, 64), None, None, i(4), good)
    with pytest.raises(ValueError, match="are needed"):
        api.paged_append_rotary(None, b(4, 2, 64), b(4, 2, 64), i(4), None, i(4), kv, kv)
    with pytest.raises(ValueError, match="cos_sin must be"):
        api.paged_append_rotary(None, b(4, 2, 64), b(4, 2, 64), i(4), cuda(torch.zeros(50)), i(4), kv, kv)
    with pytest.raises(TypeError, match="cos_sin must be torch.float32"):
        api.paged_append_rotary(None, b(4, 2, 64), b(4, 2, 64), i(4), cuda(torch.zeros(50, 64, dtype=torch.float64)), i(4), kv, kv)
    with pytest.raises(ValueError, match="positions must have shape"):
        api.paged_append_rotary(None, b(4, 2, 64), b(4, 2, 64), i(3), table, i(4), kv, kv)
    with pytest.raises(ValueError, match="q must be"):
        api.paged_append_rotary(b(4, 64), b(4, 2, 64), b(4, 2, 64), i(4), table, i(4), kv, kv)
    with pytest.raises(ValueError, match="q_out needs q"):
        api.paged_append_rotary(None, b(4, 2, 64), b(4, 2, 64), i(4), table, i(4), kv, kv, q_out=b(4, 4, 64))
    with pytest.raises(ValueError, match="v_new must have shape"):
        api.paged_append_rotary(None, b(4, 2, 64), b(4, 1, 64), i(4), table, i(4), kv, kv)
    with pytest.raises(TypeError, match="q dtype"):
        api.paged_attention_fp4(cuda(torch.zeros(4, 4, 64)), good, i(2, 3), i(3), i(2))
    with pytest.raises(TypeError, match="dtype torch.float32"):
        api.paged_read_fp4(good, i(4), torch.float32)
    for bad in (dict(max_positions=0, rotary_dim=64), dict(max_positions=4, rotary_dim=63),
                dict(max_positions=4, rotary_dim=64, inv_freq=torch.ones(31))):
        with pytest.raises(ValueError):
            api.rotary_table(**bad)


def test_rotary_table_is_formed_in_64_bits():
    from speculative_decoding_verification_25_gb300 import api
    t = api.rotary_table(131072, 64).double()
    angle = 131071.0 * 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    torch.testing.assert_close(t[131071], torch.cat([angle.cos(), angle.sin()]), rtol=0, atol=2.0 ** -25 * 1.01)
