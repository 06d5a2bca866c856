"""The oracle of shared pages and of attention over them, against small worked examples and against
the definitions evaluated another way."""
import numpy as np

from oracle import attention, pages


def test_fork_worked_example():
    # 10 tokens in pages of 4: two whole pages shared, the third copied to page 9
    table = [[5, 2, 7, -1], [-1, -1, -1, -1], [-1, -1, -1, -1]]
    t, s, src, dst, counts = pages.fork([0, 0], [2, 1], [10, 8], table, 4, [0] * 10, [9, 3])
    assert t.tolist() == [[5, 2, 7, -1], [5, 2, -1, -1], [5, 2, 9, -1]]
    assert s.tolist() == [0, 0, 2, 0, 0, 2, 0, 0, 0, 0]
    assert src.tolist() == [7, -1] and dst.tolist() == [9, -1] and counts.tolist() == [1, 1]


def test_free_worked_example():
    table = [[5, 2, 7], [5, 2, 9], [5, 2, -1]]
    shares = [0, 0, 2, 0, 0, 2, 0, 0, 0, 0]
    t, s, freed, n = pages.free([1], [10], table, 4, shares, 3)
    assert freed.tolist() == [9, -1, -1] and n.tolist() == [1]
    assert s.tolist() == [0, 0, 1, 0, 0, 1, 0, 0, 0, 0] and t[1].tolist() == [-1, -1, -1]
    t, s, freed, n = pages.free([0, 2, 0], [10, 8, 10], t, 4, s, 2)
    assert freed.tolist() == [2, 5] and n.tolist() == [3] and not s.any() and (t == -1).all()


def test_compact_worked_example():
    # live 1, 6, 8: three pages, so 6 and 8 move to 0 and 2
    t, s, src, dst, n = pages.compact([8, 0, 8], [[8, 1], [3, 3], [6, 1]], 4,
                                      [0, 1, 0, 0, 0, 0, 0, 0, 0], 4)
    assert t.tolist() == [[2, 1], [3, 3], [0, 1]] and s.tolist() == [0, 1, 0, 0, 0, 0, 0, 0, 0]
    assert src.tolist() == [6, 8, -1, -1] and dst.tolist() == [0, 2, -1, -1]
    assert n.tolist() == [3, 2]


def test_fork_then_free_gives_everything_back():
    g = np.random.default_rng(3)
    table = np.full((9, 6), -1)
    table[0] = g.permutation(40)[:6]
    free = [x for x in range(40) if x not in set(table[0].tolist())]
    t, s, src, dst, _ = pages.fork([0] * 8, range(1, 9), g.integers(1, 25, 8), table, 4, [0] * 40,
                                   free)
    _, s, freed, n = pages.free(range(1, 9), [24] * 8, t, 4, s, 40)
    assert not s.any()
    assert sorted(freed[:int(n[0])].tolist()) == sorted(x for x in dst.tolist() if x >= 0)


def _batch(g, kv=2, H=4, d=8, block=4):
    table = np.array([[3, 9, 4, 1], [3, 9, 6, -1], [3, 9, 0, 2]])
    k, v = g.normal(size=(2, 10, kv, block, d))
    return g.normal(size=(3, 2, H, d)), k, v, table, np.array([15, 11, 13])


def test_shared_decode_is_decode_where_the_tables_agree():
    g = np.random.default_rng(4)
    q, k, v, table, lens = _batch(g)
    for cu, prefix in (([0, 3], [8]), ([0, 3], [5]), ([1, 3], [8]), ([0, 2, 3], [8, 4]), ([0], [])):
        got = pages.shared_decode(q, k, v, table, lens, cu, prefix, 0.3)
        want = attention.paged_decode(q, k, v, table, lens, 0.3)
        for a, b in zip(got, want):
            assert np.allclose(a, b, rtol=1e-12, atol=1e-14)


def test_prefill_of_the_newest_tokens_is_decode():
    g = np.random.default_rng(5)
    q, k, v, table, lens = _batch(g)
    got = pages.prefill(q.reshape(6, 4, 8), k, v, table, [0, 2, 4, 6], lens, 0.3)
    want = attention.paged_decode(q, k, v, table, lens, 0.3)
    for a, b in zip(got, want):
        assert np.allclose(a, b.reshape(a.shape), rtol=1e-12, atol=1e-14)


def test_prefill_in_chunks_is_one_prefill():
    g = np.random.default_rng(6)
    k, v = g.normal(size=(2, 10, 2, 4, 8))
    table, q = np.array([[3, 9, 4, 1]]), g.normal(size=(15, 4, 8))
    whole = pages.prefill(q, k, v, table, [0, 15], [15], 0.5)[0]
    parts = [pages.prefill(q[a:z], k, v, table, [0, z - a], [z], 0.5)[0]
             for a, z in ((0, 6), (6, 7), (7, 15))]
    assert np.allclose(whole, np.concatenate(parts), rtol=1e-12, atol=1e-14)
    assert np.allclose(whole[0, 0], v[3, 0, 0])  # the first token sees itself
