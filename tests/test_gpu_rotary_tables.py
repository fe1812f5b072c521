"""The appends with tables that are no cosines and sines of magnitude 1: scaled ones."""
import numpy as np
import pytest

from oracle import paged_fp4 as oracle
from test_gpu_rotary import DEV, Case, _bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [2.0 ** -12, 1.0, 1.4375, 5.0, 2.0 ** 10, 2.0 ** 40])
@pytest.mark.parametrize("interleaved", [False, True])
def test_codes_are_exact_for_tables_of_any_size(size, interleaved):
    """Pairs that nearly cancel in one of their two results, so that float32's error is large
    beside it: every code and scale is that of exact arithmetic."""
    import torch
    from speculative_decoding_verification_25_gb300 import api
    c = Case(1500, 0, 8, 128, 128, interleaved, 64, "bf16", seed=1, far=512)
    g = torch.Generator().manual_seed(3)
    for x in (c.k_new, c.v_new):
        x.copy_((1 + torch.randint(-3, 4, x.shape, generator=g) / 128).to(torch.bfloat16))
    c.table = (size * (1 + (torch.rand(512, 128, generator=g) - 0.5) * 2.0 ** -7)).to(DEV)
    gain = float(2.0 ** np.floor(np.log2(size)) / 64)
    for gains in ((gain, 1.0), (gain * 1.203125, 0.3)):
        gains = tuple(float(np.float32(x)) for x in gains)
        cache = c.random_cache_fp4()
        want = [_bits(t).copy() for t in cache]
        api.paged_append_fp4(None, c.k_new, c.v_new, c.positions, c.table, c.slots, cache, k_gain=gains[0],
                             v_gain=gains[1], interleaved=interleaved)
        good = np.array([t for t, s in enumerate(c.slots.tolist()) if s >= 0])
        slots = c.slots.cpu().numpy()[good]
        for i, (x, gain_i) in enumerate(((c.turned(c.k_new), gains[0]), (c.host(c.v_new), gains[1]))):
            codes, scales = oracle.encode(x[good], gain_i)
            want[2 * i][slots // c.page, :, slots % c.page] = codes
            want[2 * i + 1][slots // c.page, :, slots % c.page] = scales
        for name, t, w in zip(cache._fields, cache, want):
            np.testing.assert_array_equal(_bits(t), w, err_msg=name)
