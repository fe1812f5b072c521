"""Pins of the 4-bit cache's oracle: by hand, and against torch's own e4m3."""
import numpy as np
import pytest
import torch

from oracle import paged_fp4 as oracle


def test_formats_by_hand():
    assert oracle.FOURS.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    eights = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(oracle.EIGHTS, eights)
    assert np.isnan(torch.tensor(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().item())


def test_ties_go_to_the_even_code():
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 100.0])
    assert oracle.nearest(ties, oracle.FOURS).tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 7]
    assert oracle.nearest(np.nextafter(ties, 9)[:7], oracle.FOURS).tolist() == [1, 2, 3, 4, 5, 6, 7]
    assert oracle.nearest(np.nextafter(ties, 0)[:7], oracle.FOURS).tolist() == [0, 1, 2, 3, 4, 5, 6]


def test_scales_round_as_torch_rounds():
    x = torch.rand(20000, generator=torch.Generator().manual_seed(1)).mul(440)
    x[::3] *= 2.0 ** -12
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(oracle.nearest(x.double().numpy(), oracle.EIGHTS), want)


def test_a_group_by_hand():
    x = np.zeros((1, 32))
    x[0, :4] = 12, -6, 1.1, -0.3
    codes, scales = oracle.encode(x)
    assert scales.tolist() == [[64, 0]]                       # 12 / 6 = 2, and nothing
    assert codes[0, :2].tolist() == [7 | 13 << 4, 1 | 8 << 4]   # 6, -3, 0.5, -0 times 2
    np.testing.assert_array_equal(oracle.decode(codes, scales)[0, :5], [12, -6, 1, 0, 0])
    np.testing.assert_array_equal(oracle.decode(*oracle.encode(x, 0.25), 0.25)[0, :4], [12, -6, 1, 0])


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_groups_that_are_not_finite_are_nan(bad):
    x = np.full((2, 32), 6.0)
    x[1, 20] = bad
    y = oracle.decode(*oracle.encode(x))
    assert np.isnan(y[1, 16:]).all() and (y[0] == 6).all() and (y[1, :16] == 6).all()


@pytest.mark.parametrize("gain", [1.0, 0.1015625, 64.0])
def test_values_are_within_half_a_step(gain):
    x = np.random.default_rng(3).normal(size=(500, 128)) * np.exp(np.random.default_rng(4).normal(size=(500, 1)))
    y = oracle.decode(*oracle.encode(x, gain), gain)
    top = np.abs(x.reshape(500, 8, 16)).max(-1, keepdims=True).repeat(16, -1).reshape(x.shape)
    # codes lie up to 2 apart, the largest magnitude is at most 6 (1 + 1/16) of a scale's step
    assert (np.abs(x - y) <= top / 6 * (1 + 2.0 ** -4) + 2.0 ** -10 * 6 * gain).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_turns_pairs(interleaved):
    rng = np.random.default_rng(0)
    x = rng.normal(size=(3, 2, 64))
    angle = rng.normal(size=(5, 16))
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    y = oracle.rotate(x, [4, -1, 0], table, interleaved)
    assert (y[1] == 0).all()
    np.testing.assert_array_equal(y[[0, 2], :, 32:], x[[0, 2], :, 32:])
    np.testing.assert_allclose((y[0] ** 2).sum(-1), (x[0] ** 2).sum(-1))
    a, b = (2, 3) if interleaved else (1, 17)
    turned = (x[0, 0, a] + 1j * x[0, 0, b]) * np.exp(1j * angle[4, 1])
    np.testing.assert_allclose([y[0, 0, a], y[0, 0, b]], [turned.real, turned.imag])
