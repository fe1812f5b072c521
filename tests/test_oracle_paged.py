"""Pins of the paged cache oracle: small examples by hand, and attention
against differences of a potential and against a mask written out."""
import numpy as np
import pytest

from oracle import paged


def test_plan_takes_given_back_pages_first_then_the_top_of_the_stack():
    table = np.array([[4, 5, 6, 0], [7, 0, 0, 0], [8, 9, 0, 0]], np.int32)
    r = paged.plan([8, 7, 16], [1, 10, 1], [3, 1, 2], table, [1, 2, 3], 8, 16)
    # row 0 wants 2 of its 3 pages: 6 comes back; row 1 wants 2 more: 6, then 3; row 2 wants one: 2
    assert r.cu_new.tolist() == [0, 1, 11, 12]
    assert r.block_table.tolist() == [[4, 5, 6, 0], [7, 6, 3, 0], [8, 9, 2, 0]]
    assert r.page_count.tolist() == [2, 3, 3] and r.stack == [1]
    assert r.kv_len.tolist() == [9, 17, 17]
    assert r.slot_map.tolist() == [40, 63] + list(range(48, 56)) + [24, 16] + [-1] * 4
    assert r.positions.tolist() == [8, *range(7, 17), 16] + [-1] * 4


def test_giving_back_restores_the_stack():
    stack = [10, 11, 12, 13, 14, 15]
    table = np.zeros((3, 4), np.int32)
    table[:, 0] = [1, 2, 3]
    up = paged.plan([8, 8, 8], [9, 8, 17], [1, 1, 1], table, stack, 8, 64)
    down = paged.plan([8, 8, 8], [0, 0, 0], up.page_count, up.block_table, up.stack, 8, 64)
    assert down.stack == stack and down.page_count.tolist() == [1, 1, 1]


def test_rows_that_are_not_served():
    table = np.zeros((5, 2), np.int32)
    r = paged.plan([0, 0, -1, 0, 0], [8, 16, 1, 8, 9], [0, 0, 0, 0, 0], table, [3, 4], 8, 32)
    assert r.kv_len.tolist() == [8, 0, 0, 0, 0]       # one page left for a row that wants two
    assert r.cu_new.tolist() == [0, 8, 24, 24, 32, 32]   # 9 more do not fit 32
    assert (r.slot_map[8:] == -1).all() and r.positions[8:24].tolist() == list(range(16))
    assert r.no_pages and r.clipped and r.bad_length and r.stack == [3]


def test_append_copies_tokens_to_their_slots():
    rng = np.random.default_rng(0)
    new = rng.normal(size=(3, 2, 4))
    k, v = paged.append(new, -new, [9, -1, 0], np.zeros((2, 2, 8, 4)), np.zeros((2, 2, 8, 4)))
    np.testing.assert_array_equal(k[1, :, 1], new[0])
    np.testing.assert_array_equal(v[0, :, 0], -new[2])
    assert np.count_nonzero(k) == 16


@pytest.mark.parametrize("L,n", [(5, 1), (6, 3), (4, 4), (2, 4)])
def test_attention_is_the_gradient_of_its_normaliser(L, n):
    """d lse / d q = scale * sum_j softmax_j k_j, which is attention with the
    keys as values; the causal mask written out as a list of visible keys."""
    rng = np.random.default_rng(L * 8 + n)
    D, page, scale = 6, 2, 0.4
    k = rng.normal(size=(4, 1, page, D))
    table = np.array([[2, 0, 3]])
    q = rng.normal(size=(n, 2, D))
    run = lambda x: paged.attention(x, k, k, table, [0, n], [L], scale, "f16")
    r = run(q)
    keys = k[[2, 0, 3], 0].reshape(-1, D)
    for i in range(n):
        visible = [j for j in range(L) if j <= L - n + i]
        if not visible:
            assert (r.out[i] == 0).all() and np.isneginf(r.lse[i]).all()
            continue
        for h in range(2):
            x = np.array([scale * q[i, h] @ keys[j] for j in visible])
            assert abs(np.log(np.exp(x).sum()) - r.lse[i, h]) < 1e-12
            for d in range(D):
                step = np.zeros_like(q)
                step[i, h, d] = 1e-5
                slope = (run(q + step).lse[i, h] - run(q - step).lse[i, h]) / 2e-5
                assert abs(slope - scale * r.out[i, h, d]) < 1e-8


def test_page_size_does_not_matter():
    rng = np.random.default_rng(3)
    kv = rng.normal(size=(2, 8, 1, 4))
    q = rng.normal(size=(3, 2, 4))
    whole = paged.attention(q, *(x.transpose(1, 0, 2)[None] for x in kv), np.array([[0]]), [0, 3], [7], 1.0, "bf16")
    pages = paged.attention(q, *(x.reshape(4, 2, 1, 4).transpose(0, 2, 1, 3) for x in kv), np.array([[0, 1, 2, 3]]),
                            [0, 3], [7], 1.0, "bf16")
    np.testing.assert_allclose(whole.out, pages.out, rtol=1e-13)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_bounds_admit_one_rounding_of_probabilities_and_results(dtype):
    """Exact arithmetic that rounds the probabilities once and the result once
    stays inside the bounds, on few keys, where nothing averages out."""
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float16
    rounded = lambda x: torch.from_numpy(x).to(dt).double().numpy()
    rng = np.random.default_rng(7)
    worst = 0.0
    for L in (1, 2, 3, 5, 8):
        for _ in range(60):
            q, k, v = (rounded(rng.normal(size=s)) for s in ((1, 4, 64), (1, 1, L, 64), (1, 1, L, 64)))
            r = paged.attention(q, k, v, np.array([[0]]), [0, 1], [L], 0.125, dtype)
            x = q[0] @ k[0, 0].T * 0.125
            w = np.exp(x - x.max(-1, keepdims=True))
            o = rounded(rounded(w) @ v[0, 0] / w.sum(-1, keepdims=True))
            worst = max(worst, float((np.abs(o - r.out[0]) / r.out_tol[0]).max()))
    assert 0.4 < worst <= 1, worst
