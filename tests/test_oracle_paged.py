"""The paged-cache oracle against second formulations: numpy softmax over
gathered tokens, complex rotations, differences of the forward pass, and page
operations worked out by hand."""
import numpy as np
import pytest

from paged_util import random_table


def test_attention_is_softmax_over_the_gathered_tokens(orc):
    rng = np.random.default_rng(1)
    lens, slots, heads, group, depth = [0, 1, 7, 12, 40], 5, 2, 3, 9
    table = random_table(rng, lens, slots, 14, 8)
    table[3, 1] = -1   # a hole
    table[4, 2] = 14   # past the pool
    k, v = rng.standard_normal((2, 14, slots, heads, depth))
    q = rng.standard_normal((5, heads * group, depth))
    for window in (0, 6):
        out, lse, abs_out, _ = orc.paged_attention(q, k, v, table, lens, 0.3, window)
        for b, n in enumerate(lens):
            js = [j for j in range(max(0, n - window) if window else 0, n) if 0 <= table[b, j // slots] < 14]
            for h in range(heads * group):
                if not js:
                    assert np.all(out[b, h] == 0) and lse[b, h] == -np.inf
                    continue
                kk = np.stack([k[table[b, j // slots], j % slots, h // group] for j in js])
                vv = np.stack([v[table[b, j // slots], j % slots, h // group] for j in js])
                e = np.exp(0.3 * kk @ q[b, h])
                np.testing.assert_allclose(out[b, h], e @ vv / e.sum(), rtol=1e-12, atol=1e-14)
                np.testing.assert_allclose(abs_out[b, h], e @ np.abs(vv) / e.sum(), rtol=1e-12)
                np.testing.assert_allclose(lse[b, h], np.log(e.sum()), rtol=1e-12, atol=1e-14)


def test_attention_clamps_lengths_to_the_table(orc):
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 4, 3, 1, 8))
    q = rng.standard_normal((2, 1, 8))
    table = np.array([[0, 1], [2, 3]], dtype=np.int32)
    a = orc.paged_attention(q, k, v, table, [6, 0], 1.0)
    b = orc.paged_attention(q, k, v, table, [100, -4], 1.0)
    for x, y in zip(a, b):
        np.testing.assert_array_equal(x, y)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [0, 6, 10])
def test_norm_rope_is_a_complex_rotation(orc, interleaved, rotary):
    rng = np.random.default_rng(3)
    x, w = rng.standard_normal((4, 3, 10)), rng.standard_normal(10)
    pos = np.array([0, 1, -7, 123456], dtype=np.int32)
    f = rng.random(rotary // 2).astype(np.float32)
    y, bound = orc.norm_rope(x, w, pos, f, interleaved, 1.25, True, 1e-5)
    n = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + 1e-5) * w
    a = np.arange(rotary // 2) * (2 if interleaved else 1)
    b = a + (1 if interleaved else rotary // 2)
    z = (n[..., a] + 1j * n[..., b]) * 1.25 * np.exp(1j * pos[:, None, None].astype(np.float64) * f.astype(np.float64))
    want = n.copy()
    want[..., a], want[..., b] = z.real, z.imag
    np.testing.assert_allclose(y, want, rtol=1e-9, atol=1e-9)
    assert np.all(bound >= np.abs(y) * (1 - 1e-12))
    plain, _ = orc.norm_rope(x, None, pos, f, interleaved, 1.0, False)
    np.testing.assert_allclose((plain ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-12)  # a rotation keeps lengths


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_backward_is_the_derivative(orc, norm, interleaved):
    """Central differences of L = sum dy . y in every input and weight."""
    rng = np.random.default_rng(4)
    x, dy, w = rng.standard_normal((2, 2, 6)), rng.standard_normal((2, 2, 6)), 1 + 0.3 * rng.standard_normal(6)
    pos, f = np.array([3, 11], dtype=np.int32), np.array([1.0, 0.1], dtype=np.float32)
    w = w if norm else None
    args = (pos, f, interleaved, 1.1, norm, 1e-3)
    loss = lambda x, w: (orc.norm_rope(x, w, *args)[0] * dy).sum()  # noqa: E731
    dx, _, dw, _ = orc.norm_rope_backward(dy, x, w, *args)
    h = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    if norm:
        for i in range(6):
            e = np.zeros(6)
            e[i] = h
            assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_page_operations_by_hand(orc):
    cache = np.arange(2 * 6 * 2, dtype=np.int32).reshape(2, 6, 2)
    was = cache.copy()
    table = np.array([[4, 2, -1], [-1, -1, -1], [5, -1, -1]], dtype=np.int32)
    lens, refs = np.array([5, 0, 3], np.int32), np.array([0, 0, 1, 0, 1, 1], np.int32)
    # row 0 holds 5 tokens in pages of 3: page 4 is full, page 2 is not
    assert orc.pages_fork(cache, table, lens, refs, 3, [0], [1]) == 0
    np.testing.assert_array_equal(table, [[4, 2, -1], [4, 0, -1], [5, -1, -1]])
    np.testing.assert_array_equal(refs, [1, 0, 1, 0, 2, 1])
    np.testing.assert_array_equal(lens, [5, 5, 3])
    np.testing.assert_array_equal(cache[:, 0], was[:, 2])
    orc.pages_free(table, lens, refs, [0, 0, 7])
    np.testing.assert_array_equal(table[0], [-1, -1, -1])
    np.testing.assert_array_equal(refs, [1, 0, 0, 0, 1, 1])
    # live pages 0, 4, 5: 4 -> 1, 5 -> 2
    was = cache.copy()
    remap = orc.pages_compact(cache, table, refs)
    np.testing.assert_array_equal(remap, [0, -1, -1, -1, 1, 2])
    np.testing.assert_array_equal(table, [[-1, -1, -1], [1, 0, -1], [2, -1, -1]])
    np.testing.assert_array_equal(refs, [1, 1, 1, 0, 0, 0])
    np.testing.assert_array_equal(cache[:, [1, 2]], was[:, [4, 5]])
    # row 0 wants two pages, row 1 has room for one more token, row 2 wants two pages and finds one
    assert orc.pages_reserve(table, lens, np.array([4, 1, 7], np.int32), refs, 3) == 1
    np.testing.assert_array_equal(table, [[3, 4, -1], [1, 0, -1], [2, 5, -1]])
    np.testing.assert_array_equal(refs, [1] * 6)
