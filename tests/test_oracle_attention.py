"""The fp64 attention reference against what can be said without it: closed forms, and the two
forms of latent attention against each other and against plain multi-head attention."""
import numpy as np
import pytest

from oracle import attention as ref


def rng(seed):
    return np.random.default_rng(seed)


def table_for(lens, block, extra=1):
    need = [-(-n // block) for n in lens]
    width = max(need) + extra
    t = np.full((len(lens), width), -1, dtype=np.int32)
    ids = rng(7).permutation(sum(need) + 2)
    at = 0
    for i, k in enumerate(need):
        t[i, :k] = ids[at:at + k]
        at += k
    return t, sum(need) + 2


def test_equal_keys_give_the_mean_of_the_visible_values():
    g = rng(0)
    lens, block = [11, 4, 0], 4
    table, n = table_for(lens, block)
    k = np.ones((n, 2, block, 8))
    v = g.normal(size=k.shape)
    q = g.normal(size=(3, 2, 4, 8))
    o, mag, top = ref.paged_decode(q, k, v, table, lens, 0.3)
    for b in range(3):
        for p in range(2):
            seen = max(lens[b] - 1 + p, 0)
            for h in range(4):
                rows = np.array([v[table[b, j // block], h // 2, j % block] for j in range(seen)])
                want = rows.mean(axis=0) if seen else np.zeros(8)
                np.testing.assert_allclose(o[b, p, h], want, atol=1e-14)
                np.testing.assert_allclose(mag[b, p, h], np.abs(rows).mean(axis=0) if seen
                                           else np.zeros(8), atol=1e-14)
    assert top.max() <= 0.3 * np.abs(q).sum(-1).max() + 1e-12


def test_a_dominant_key_gives_its_value_and_null_pages_are_not_seen():
    block, d = 3, 4
    table = np.array([[2, -1, 0, 7]], dtype=np.int32)  # 7 is no page either
    k = np.zeros((3, 1, block, d))
    v = rng(1).normal(size=k.shape)
    k[0, 0, 1] = 50.0                                  # position 7
    q = np.ones((1, 1, 1, d))
    o, _, _ = ref.paged_decode(q, k, v, table, [12], 1.0)
    np.testing.assert_allclose(o[0, 0, 0], v[0, 0, 1], atol=1e-12)
    seen = ref.visible(table[0], 12, block, 3)
    assert [x[0] for x in seen] == [0, 1, 2, 6, 7, 8]
    assert ref.visible(table[0], 2, block, 3) == [(0, 2, 0), (1, 2, 1)]
    assert ref.visible(table[0], -4, block, 3) == []


def test_scores_move_all_alike_without_changing_the_output():
    g = rng(2)
    k, v, q = g.normal(size=(9, 6)), g.normal(size=(9, 5)), g.normal(size=6)
    base, _, _ = ref.attend(q, k, v, 0.7)
    shifted = k + 1000.0 * q / (q @ q) / 0.7           # every score + 1000
    np.testing.assert_allclose(ref.attend(q, shifted, v, 0.7)[0], base, rtol=1e-9)
    np.testing.assert_allclose(ref.attend(-q, k, v, -0.7)[0], base, rtol=1e-12)
    np.testing.assert_allclose(ref.attend(q, k, v, 0.0)[0], v.mean(axis=0), rtol=1e-12)


def test_derivative_of_the_output_by_a_value_is_its_weight():
    g = rng(3)
    k, v, q = g.normal(size=(6, 4)), g.normal(size=(6, 3)), g.normal(size=4)
    s = 0.4 * (k @ q)
    p = np.exp(s) / np.exp(s).sum()
    for j in range(6):
        up = v.copy()
        up[j] += 1.0
        np.testing.assert_allclose(ref.attend(q, k, up, 0.4)[0] - ref.attend(q, k, v, 0.4)[0],
                                   np.full(3, p[j]), rtol=1e-12)


@pytest.mark.parametrize("scale", [0.2, -0.3, 0.0])
def test_absorbed_expanded_and_plain_attention_agree(scale):
    g = rng(4)
    lens, new, block, H, R, rope, dn = [9, 5, 1], [4, 5, 1], 4, 3, 16, 6, 8
    table, n = table_for(lens, block)
    cache = g.normal(size=(n, block, R + rope))
    w = g.normal(size=(H, 2 * dn, R)) / 4
    cu = np.cumsum([0] + new)
    qn, qp = g.normal(size=(cu[-1], H, dn)), g.normal(size=(cu[-1], H, rope))
    got = ref.latent_expanded(qn, qp, w, cache, table, cu, lens, scale)
    for i in range(3):
        a = slice(cu[i], cu[i + 1])
        np.testing.assert_allclose(
            ref.latent_absorbed(qn[None, a], qp[None, a], w, cache, table[i:i + 1],
                                lens[i:i + 1], scale)[0], got[a], atol=1e-12)
        # the same request with every head's keys and values in an ordinary cache
        rows = np.stack([cache[table[i, j // block], j % block] for j in range(lens[i])])
        k = np.concatenate([np.einsum("hdr,jr->hjd", w[:, :dn], rows[:, :R]),
                            np.broadcast_to(rows[:, R:], (H, lens[i], rope))], axis=2)
        v = np.pad(np.einsum("hdr,jr->hjd", w[:, dn:], rows[:, :R]), ((0, 0), (0, 0), (0, rope)))
        q = np.concatenate([qn[a], qp[a]], axis=2)[None]
        plain, _, _ = ref.paged_decode(q, k[None], v[None], np.zeros((1, 1), dtype=np.int32),
                                       [lens[i]], scale)
        np.testing.assert_allclose(plain[0, :, :, :dn], got[a], atol=1e-12)


def test_plan_hands_out_pages_in_request_order():
    table = np.array([[5, 9, 9, 9], [4, 9, 9, 9], [9, 9, 9, 9]], dtype=np.int32)
    t, cu, lens, slots, pos, counts = ref.plan([3, 4, 0], [2, 1, 5], table, [10, 11, 12, 13], 4, 10)
    assert t.tolist() == [[5, 10, 9, 9], [4, 11, 9, 9], [12, 13, 9, 9]]
    assert cu.tolist() == [0, 2, 3, 8] and lens.tolist() == [5, 5, 5]
    assert slots.tolist() == [23, 40, 44, 48, 49, 50, 51, 52, -1, -1]
    assert pos.tolist() == [3, 4, 4, 0, 1, 2, 3, 4, 0, 0]
    assert counts.tolist() == [8, 4]


def test_plan_slots_are_distinct_and_where_decode_looks():
    g = rng(6)
    block, width = 5, 12
    ctx, new = g.integers(0, 30, 8), g.integers(0, 20, 8)
    need = -(-ctx // block)
    pool = g.permutation(200).astype(np.int32)
    table = np.full((8, width), -1, dtype=np.int32)
    at = 0
    for i in range(8):
        table[i, :need[i]] = pool[at:at + need[i]]
        at += need[i]
    t, cu, lens, slots, pos, counts = ref.plan(ctx, new, table, pool[at:], block, int(new.sum()))
    assert len(set(slots.tolist())) == len(slots) and slots.min() >= 0
    assert counts[1] == sum(-(-(c + w) // block) - -(-c // block) for c, w in zip(ctx, new))
    for i in range(8):
        where = {j: p * block + o for j, p, o in ref.visible(t[i], int(lens[i]), block, 200)}
        assert len(where) == lens[i]
        for x in range(cu[i], cu[i + 1]):
            assert slots[x] == where[int(pos[x])]
