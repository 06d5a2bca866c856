"""The oracle of shared decode where requests of a group ended or hold a part of the prefix: plain
decode of each request's own row."""
import numpy as np
import pytest

from oracle import attention, pages


@pytest.mark.parametrize("lens", [[0, 11, 13], [0, 0, 9], [5, 7, 3], [0, 4, 9], [0, 0, 0]])
def test_the_prefix_comes_from_a_row_that_holds_it(lens):
    g = np.random.default_rng(7)
    H, d, kv, block = 4, 8, 2, 4
    table = np.array([[3, 9, 4, 1], [3, 9, 5, 2], [3, 9, 6, 0]])
    for i, n in enumerate(lens):
        table[i, -(-n // block):] = -1
    k, v = g.normal(size=(2, 10, kv, block, d))
    q = g.normal(size=(3, 2, H, d))
    got = pages.shared_decode(q, k, v, table, lens, [0, 3], [8], 0.3)
    want = attention.paged_decode(q, k, v, table, lens, 0.3)
    for a, b in zip(got, want):
        assert np.allclose(a, b, rtol=1e-12, atol=1e-14)
