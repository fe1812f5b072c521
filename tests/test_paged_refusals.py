"""More of what the paged cache operators and their helpers refuse on the
host, before anything reaches a GPU."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def N():
    from speculative_decoding_verification_25_gb300 import build as b
    b.build()
    from speculative_decoding_verification_25_gb300 import _native
    _native.load()
    return _native


FAKE = 0x10000   # never dereferenced: every call below fails validation first
ATTEND = dict(q=FAKE, qs=1024, kc=FAKE, vc=FAKE, dtype=1, table=FAKE, cu=FAKE, kv=FAKE, B=2, T=4, Hq=8, Hk=2, D=128, page=16,
              max_pages=9, n_pages=50, scale=0.1, out=FAKE, lse=None, ws=FAKE, wsb=0, flags=None, stream=None)


def _attend(N, **kw):
    return N.spec_paged_attention_raw(*{**ATTEND, **kw}.values())


@pytest.mark.parametrize("page", [8, 16, 64, 256])
def test_attention_refuses_tables_whose_keys_pass_31_bits_in_a_tile(N, page):
    """The kernel's key numbers run two tiles and a unit's cost past the table's last key."""
    most = (2 ** 31 - 512) // page
    assert _attend(N, page=page, max_pages=most) == N.SV_ERR_WORKSPACE       # the sizes pass
    assert _attend(N, page=page, max_pages=most + 1) == N.SV_ERR_SHAPE
    assert _attend(N, page=page, max_pages=2 ** 31 // page - 1) == N.SV_ERR_SHAPE


def test_attention_refuses_scales_that_overflow(N):
    """The kernel's scale is scale * log2(e), which has to be finite as well."""
    for scale in (1e-38, 1.0, 2e38, 2.3e38):
        assert _attend(N, scale=scale) == N.SV_ERR_WORKSPACE, scale   # the scale passes
    for scale in (2.4e38, 3e38, 3.4e38):
        assert _attend(N, scale=scale) == N.SV_ERR_SHAPE, scale


def test_capture_id_needs_a_place_for_it(N):
    assert N.load().spec_stream_capture_id(None, ctypes.POINTER(ctypes.c_uint64)()) == N.SV_ERR_NULL


def test_attention_errors_need_a_workspace_and_a_place(N):
    flags = ctypes.c_uint32(0)
    call = N.load().spec_paged_attention_device_errors
    assert call(None, None, ctypes.byref(flags)) == N.SV_ERR_NULL
    assert call(FAKE, None, ctypes.POINTER(ctypes.c_uint32)()) == N.SV_ERR_NULL
    assert call(FAKE + 8, None, ctypes.byref(flags)) == N.SV_ERR_ALIGN


class FakeCuda(torch.Tensor):
    """A host tensor that says it lies on a CUDA device."""
    index = 0
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.index))


def test_scratch_is_dense_and_on_the_device(N):
    from speculative_decoding_verification_25_gb300 import api
    dev = torch.device("cuda", 0)
    good = torch.zeros(8, 4).as_subclass(FakeCuda)
    assert api._scratch(good, "workspace", dev) == (good.data_ptr(), 128)
    for bad in (torch.zeros(8, 4), torch.zeros(8, 4).as_subclass(FakeCuda)[:, :2], None, 1 << 16):
        with pytest.raises((TypeError, ValueError), match="workspace must be"):
            api._scratch(bad, "workspace", dev)
    good.index = 1
    with pytest.raises(ValueError, match="workspace is on cuda:1"):
        api._scratch(good, "workspace", dev)
    with pytest.raises(ValueError, match="workspace"):
        api.attention_errors(torch.zeros(8192, dtype=torch.uint8))
    with pytest.raises(ValueError, match="smaller than its counters"):
        api.attention_errors(torch.zeros(64, dtype=torch.uint8).as_subclass(FakeCuda))


@pytest.mark.gpu
def test_attention_refuses_workspaces_of_the_host_and_strided_ones(N):
    from paged_util import PagedCase
    c = PagedCase([(40, 3)], 4, 2, 64, 16, "bf16")
    need = N.spec_paged_attention_workspace_bytes(64)
    with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
        c.run(workspace=torch.zeros(need, dtype=torch.uint8))
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        c.run(workspace=torch.zeros(need, 2, dtype=torch.uint8, device="cuda:0")[:, 0])
    with pytest.raises(TypeError, match="workspace"):
        c.run(workspace=12345)
    with pytest.raises(N.SpecVerifyError):
        c.run(workspace=torch.zeros(need - 16, dtype=torch.uint8, device="cuda:0"))
