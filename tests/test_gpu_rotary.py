"""The appends with a rotation and the 4-bit cache's append and read on the GPU
against the 64-bit oracle: rotated values within their rounding, copies, codes
and scales bit by bit."""
import numpy as np
import pytest

from oracle import paged as paged_oracle
from oracle import paged_fp4 as oracle
from paged_util import torch_dtype

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

#       T, Hq, Hk, D, rot, interleaved, page, dtype
SHAPES = [(1, 1, 1, 64, 32, False, 8, "bf16"), (5, 32, 8, 128, 128, False, 16, "bf16"),
          (77, 28, 4, 64, 64, True, 8, "f16"), (130, 6, 3, 128, 96, True, 32, "bf16"),
          (131, 7, 7, 128, 64, False, 256, "f16"), (64, 0, 2, 64, 32, True, 64, "bf16"),
          (300, 16, 1, 64, 64, False, 128, "bf16"), (33, 5, 5, 128, 32, False, 16, "f16")]


class Case:
    def __init__(self, T, Hq, Hk, D, rot, interleaved, page, dtype, seed=0, far=9000, spread=1.0):
        import torch
        from speculative_decoding_verification_25_gb300 import api
        g = torch.Generator().manual_seed(seed)
        dt = torch_dtype(dtype)
        self.T, self.Hq, self.Hk, self.D, self.page, self.dtype, self.interleaved = T, Hq, Hk, D, page, dtype, interleaved
        self.n_pages = -(-T // page) + 2
        self.qkv = (torch.randn(T, Hq + 2 * Hk + 1, D, generator=g) * spread).to(dt).to(DEV)
        self.q = self.qkv[:, :Hq] if Hq else None
        self.k_new, self.v_new = self.qkv[:, Hq:Hq + Hk], self.qkv[:, Hq + Hk + 1:]
        self.positions = torch.randint(0, far, (T,), generator=g).to(torch.int32)
        self.slots = torch.randperm(self.n_pages * page, generator=g)[:T].to(torch.int32)
        self.slots[1::7] = -1
        self.positions[2::11], self.slots[2::11] = -1, -1
        self.positions, self.slots = self.positions.to(DEV), self.slots.to(DEV)
        self.table = api.rotary_table(far, rot, device=DEV)
        self.flags = torch.zeros(1, dtype=torch.int32, device=DEV)

    def host(self, x):
        return x.double().cpu().numpy()

    def turned(self, x):
        return oracle.rotate(self.host(x), self.positions.tolist(), self.host(self.table), self.interleaved)

    def check_rotated(self, got, x):
        want, p = self.turned(x), self.positions.tolist()
        tol = oracle.rotation_tolerance(self.host(x), want, p, self.host(self.table), self.dtype, self.interleaved)
        assert (np.abs(self.host(got) - want) <= tol).all()

    def random_caches(self):
        import torch
        g = torch.Generator().manual_seed(99)
        shape = (self.n_pages, self.Hk, self.page, self.D)
        return [torch.randn(shape, generator=g).to(torch_dtype(self.dtype)).to(DEV) for _ in range(2)]

    def random_cache_fp4(self):
        import torch
        from speculative_decoding_verification_25_gb300 import api
        g = torch.Generator().manual_seed(98)
        cache = api.paged_cache_fp4(self.n_pages, self.Hk, self.page, self.D, DEV)
        for t in cache:
            t.view(torch.uint8).copy_(torch.randint(0, 120, t.shape, generator=g, dtype=torch.uint8))
        return cache


def _bits(t):
    import torch
    return t.view(torch.int16 if t.element_size() == 2 else torch.uint8).cpu().numpy()


@pytest.mark.parametrize("shape", SHAPES)
def test_append_rotary(shape):
    from speculative_decoding_verification_25_gb300 import api
    c = Case(*shape, seed=shape[0])
    k, v = c.random_caches()
    k0, v0 = _bits(k).copy(), _bits(v).copy()
    before = k.clone()
    q = api.paged_append_rotary(c.q, c.k_new, c.v_new, c.positions, c.table, c.slots, k, v, interleaved=c.interleaved,
                                flags=c.flags)
    assert (q is None) == (c.Hq == 0)
    if c.Hq:
        c.check_rotated(q, c.q)
    slots = c.slots.tolist()
    want = paged_oracle.append(_bits(c.k_new.contiguous()), _bits(c.v_new.contiguous()), slots, k0, v0)
    np.testing.assert_array_equal(_bits(v), want[1])
    got = k.transpose(1, 2).flatten(0, 1)
    placed = [t for t, s in enumerate(slots) if s >= 0]
    all_new = c.k_new.new_zeros(c.T, c.Hk, c.D)
    all_new[placed] = got[[slots[t] for t in placed]]
    keep = c.positions.clone()
    for t, s in enumerate(slots):
        if s < 0:
            keep[t] = -1
    c.positions = keep
    c.check_rotated(all_new, c.k_new)
    untouched = [s for s in range(c.n_pages * c.page) if s not in set(slots)]
    np.testing.assert_array_equal(_bits(got[untouched]), _bits(before.transpose(1, 2).flatten(0, 1)[untouched].contiguous()))
    assert c.flags.item() == 0


@pytest.mark.parametrize("gains", [(1.0, 1.0), (0.25, 2.0 ** -5), (0.1, 0.3)])
@pytest.mark.parametrize("shape", SHAPES)
def test_append_fp4_is_exact(shape, gains):
    """Every code and scale is that of exact arithmetic, everything else as it was."""
    from speculative_decoding_verification_25_gb300 import api
    c = Case(*shape, seed=shape[0] + 1)
    gains = tuple(float(np.float32(g)) for g in gains)
    cache = c.random_cache_fp4()
    want = [_bits(t).copy() for t in cache]
    q = api.paged_append_fp4(c.q, c.k_new, c.v_new, c.positions, c.table, c.slots, cache, k_gain=gains[0], v_gain=gains[1],
                             interleaved=c.interleaved, flags=c.flags)
    if c.Hq:
        c.check_rotated(q, c.q)
    for i, (x, gain) in enumerate(((c.turned(c.k_new), gains[0]), (c.host(c.v_new), gains[1]))):
        codes, scales = oracle.encode(x, gain)
        for t, s in enumerate(c.slots.tolist()):
            if s >= 0:
                want[2 * i][s // c.page, :, s % c.page] = codes[t]
                want[2 * i + 1][s // c.page, :, s % c.page] = scales[t]
    for name, t, w in zip(cache._fields, cache, want):
        np.testing.assert_array_equal(_bits(t), w, err_msg=name)
    assert c.flags.item() == 0


def test_append_fp4_without_a_rotation():
    import torch
    from speculative_decoding_verification_25_gb300 import api
    c = Case(50, 4, 2, 128, 128, False, 16, "bf16", seed=3)
    cache = c.random_cache_fp4()
    assert api.paged_append_fp4(None, c.k_new, c.v_new, None, None, c.slots, cache) is None
    k, v = api.paged_read_fp4(cache, c.slots, torch.bfloat16)
    for got, x in ((k, c.k_new), (v, c.v_new)):
        want = oracle.decode(*oracle.encode(c.host(x)))
        want[(c.slots < 0).cpu().numpy()] = 0
        np.testing.assert_array_equal(c.host(got), want)


def test_append_fp4_of_borders_and_extremes():
    """Values at, and one step beside, every border; groups of zeros, of tiny and
    of huge numbers, NaN and infinities; angles whose sines and cosines cancel."""
    import torch
    from speculative_decoding_verification_25_gb300 import api
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 1.5, 3.0, 0.0])
    for dtype in ("bf16", "f16"):
        c = Case(64, 2, 2, 64, 64, False, 8, dtype, seed=5)
        x = torch.zeros(64, 16)
        for i in range(64):
            x[i] = borders[torch.randint(0, 11, (16,), generator=torch.Generator().manual_seed(i))] * 2.0 ** (i % 13 - 6) * (1 + i % 8 / 8)
            x[i, 3] = 6 * 2.0 ** (i % 13 - 6) * (1 + i % 8 / 8)
            x[i, ::2] *= -1
        beside = x.to(torch_dtype(dtype)).view(torch.int16) + torch.randint(-1, 2, x.shape, generator=torch.Generator().manual_seed(7)).to(torch.int16)
        x[::3] = beside.view(torch_dtype(dtype)).float()[::3]
        for i, special in enumerate((float("nan"), float("inf"), -float("inf"))):
            x[50 + i, 9] = special
        x[55], x[56], x[57], x[58] = 0.0, 2.0 ** -20, 60000.0, 2.0 ** -12
        c.k_new[:, 0] = x.repeat(1, 4).to(torch_dtype(dtype)).to(DEV)
        c.v_new[:, 1] = x.flip(1).repeat(1, 4).to(torch_dtype(dtype)).to(DEV)
        # exact turns (cosines and sines of 0, 1 and -1) and turns by about a quarter of pi
        c.table[:] = 0
        c.table[0::3, :32] = 1
        c.table[1::3, 32:] = -1
        c.table[2::3, :32], c.table[2::3, 32:] = 0.70710678, 0.70710677
        c.positions = torch.arange(64, dtype=torch.int32, device=DEV)
        c.slots = torch.arange(64, dtype=torch.int32, device=DEV)
        for rotated in (True, False):
            cache = c.random_cache_fp4()
            api.paged_append_fp4(None, c.k_new, c.v_new, c.positions if rotated else None, c.table if rotated else None,
                                 c.slots, cache)
            with np.errstate(invalid="ignore"):
                k = c.turned(c.k_new) if rotated else c.host(c.k_new)
            for i, want in enumerate((k, c.host(c.v_new))):
                codes, scales = oracle.encode(want)
                got = [_bits(t.view(torch.uint8).transpose(1, 2).flatten(0, 1)[:64].contiguous()) for t in cache[2 * i:2 * i + 2]]
                np.testing.assert_array_equal(got[1], scales)
                np.testing.assert_array_equal(got[0], codes)


@pytest.mark.parametrize("T,Hk,D,page,dtype", [(1, 1, 64, 8, "bf16"), (333, 3, 128, 32, "f16"), (2049, 8, 64, 256, "bf16")])
def test_read_fp4(T, Hk, D, page, dtype):
    import torch
    from speculative_decoding_verification_25_gb300 import _native as N, api
    c = Case(T, 1, Hk, D, 32, False, page, dtype, seed=T)
    cache = c.random_cache_fp4()
    slots = c.slots.clone()
    slots[T // 2] = slots[0]             # the same slot twice
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    for gains in ((1.0, 1.0), (0.125, 0.3)):
        k, v = api.paged_read_fp4(cache, slots, torch_dtype(dtype), k_gain=gains[0], v_gain=gains[1], flags=flags)
        for got, codes, scales, gain in ((k, cache.k, cache.k_scale, gains[0]), (v, cache.v, cache.v_scale, gains[1])):
            want = oracle.decode(_bits(codes), _bits(scales), gain).transpose(0, 2, 1, 3).reshape(-1, Hk, D)[slots.clamp(min=0).cpu().numpy()]
            want[(slots < 0).cpu().numpy()] = 0
            u, tiny = paged_oracle.UNIT[dtype]
            # the gain's own rounding to float32, the product's, and the result's
            assert (np.abs(c.host(got) - want) <= (u + 3 * 2.0 ** -24) * np.abs(want) + tiny).all()
    assert flags.item() == 0
    api.paged_read_fp4(cache, torch.tensor([c.n_pages * page], dtype=torch.int32, device=DEV), flags=flags)
    assert flags.item() == N.SV_DEV_BAD_PAGE


def test_positions_and_slots_that_are_none():
    import torch
    from speculative_decoding_verification_25_gb300 import _native as N, api
    c = Case(6, 2, 1, 64, 32, False, 8, "bf16", far=40)
    c.positions.copy_(torch.tensor([3, 40, -1, 39, 2 ** 31 - 1, -5]))
    c.slots.copy_(torch.tensor([0, 1, -1, 2, 3, 4]))
    for fp4 in (False, True):
        k, v = c.random_caches()
        cache = c.random_cache_fp4()
        before = [_bits(t).copy() for t in (cache if fp4 else (k, v))]
        c.flags.zero_()
        if fp4:
            q = api.paged_append_fp4(c.q, c.k_new, c.v_new, c.positions, c.table, c.slots, cache, flags=c.flags)
        else:
            q = api.paged_append_rotary(c.q, c.k_new, c.v_new, c.positions, c.table, c.slots, k, v, flags=c.flags)
        assert c.flags.item() == N.SV_DEV_BAD_LENGTH
        assert float(q[[1, 2, 4, 5]].abs().sum()) == 0 and float(q[[0, 3]].abs().sum()) > 0
        for t, b in zip(cache if fp4 else (k, v), before):
            same = (_bits(t) == b).reshape(c.n_pages, c.Hk, c.page, -1).all((1, 3)).ravel()
            assert not same[0] and not same[2] and same[[1, 3, 4, 5, 6, 7]].all()
        c.flags.zero_()
        slots = c.slots.clone()
        slots[0] = c.n_pages * c.page
        if fp4:
            api.paged_append_fp4(None, c.k_new, c.v_new, None, None, slots, cache, flags=c.flags)
        else:
            api.paged_append_rotary(None, c.k_new, c.v_new, c.positions.clamp(0, 39), c.table, slots, k, v, flags=c.flags)
        assert c.flags.item() == N.SV_DEV_BAD_PAGE


def test_queries_rotated_in_place():
    from speculative_decoding_verification_25_gb300 import api
    c = Case(41, 9, 3, 128, 64, True, 16, "bf16", seed=8)
    k, v = c.random_caches()
    x = c.q.clone()
    apart = api.paged_append_rotary(c.q, c.k_new, c.v_new, c.positions, c.table, c.slots, k, v, interleaved=True)
    here = api.paged_append_rotary(c.q, c.k_new, c.v_new, c.positions, c.table, c.slots, k, v, interleaved=True, q_out=c.q)
    assert here is c.q
    np.testing.assert_array_equal(_bits(c.q.contiguous()), _bits(apart))
    c.check_rotated(here, x)


def test_rotary_table_of_far_positions():
    import torch
    from speculative_decoding_verification_25_gb300 import api
    t = api.rotary_table(131072, 64, base=500000.0).double()
    angle = 131071 * 500000.0 ** (-np.arange(0, 64, 2) / 64)
    np.testing.assert_allclose(t[131071, :32].numpy(), np.cos(angle), rtol=0, atol=2.0 ** -25 * 1.01)
    rates = torch.tensor([1.0, 0.5])
    np.testing.assert_allclose(api.rotary_table(9, 4, inv_freq=rates)[8].double().numpy(),
                               [np.cos(8), np.cos(4), np.sin(8), np.sin(4)], rtol=0, atol=2.0 ** -25)
