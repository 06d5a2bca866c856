"""Pages that requests share: fork, free, compact and copy against the plain loops of the oracle
(whole numbers, so equal), at the sizes where both forms of each call run."""
import numpy as np
import pytest
import torch

from attn_util import gen
from gpu_util import DEV, say
from oracle import pages as oracle_pages

pytestmark = pytest.mark.gpu


def ints(values):
    return torch.tensor(np.asarray(values), dtype=torch.int32, device=DEV)


def same(got, want, what):
    for i, (a, b) in enumerate(zip(got, want)):
        a = a.cpu().numpy()
        assert a.shape == np.asarray(b).shape and np.array_equal(a, b), f"{what}: output {i}"


def shared_table(seed, rows, lens_hi, block, pool, extra_cols=2):
    """A table in which every second row shares whole pages with the row before: (table, lens,
    shares)."""
    g = np.random.default_rng(seed)
    lens = g.integers(0, lens_hi + 1, rows)
    width = max(-(-int(lens.max()) // block), 1) + extra_cols
    ids = g.permutation(pool)
    table, shares, at = np.full((rows, width), -1), np.zeros(pool, dtype=np.int64), 0
    for i in range(rows):
        need = -(-int(lens[i]) // block)
        common = 0
        if i % 2:
            common = int(g.integers(0, min(lens[i] // block, -(-int(lens[i - 1]) // block)) + 1))
        table[i, :common] = table[i - 1, :common]
        shares[table[i, :common]] += 1
        table[i, common:need] = ids[at:at + need - common]
        at += need - common
    assert at <= pool
    return table, lens, shares, [int(x) for x in ids[at:]]


# (rows, forks, block, tokens, page list too short, null entries)
@pytest.mark.parametrize("rows,forks,block,hi,short,null", [
    (2, 1, 16, 100, 0, False), (9, 5, 1, 20, 0, False), (60, 40, 24, 3000, 0, False),
    (60, 40, 24, 3000, 11, True), (700, 600, 7, 400, 0, True), (20, 19, 2, 5000, 3, False),
])
def test_fork(gpu_lib, rows, forks, block, hi, short, null):
    say("fork", rows, forks, block, hi)
    g = np.random.default_rng(rows * 7 + forks)
    parents = rows - forks
    width = -(-hi // block) + 1
    pool = parents * width + forks + 9
    ids = g.permutation(pool)
    table = np.full((rows, width), -1)
    place = g.permutation(rows)
    lens = g.integers(1, hi + 1, parents)
    at = 0
    for i in range(parents):
        need = -(-int(lens[i]) // block)
        table[place[i], :need] = ids[at:at + need]
        at += need
    if null:
        table[place[0], ::3] = -1
        table[place[0], 1] = pool + 3
    free = ids[at:at + forks - short] if short else ids[at:]
    who = g.integers(0, parents, forks)
    flen = np.array([g.integers(0, lens[i] + 1) for i in who])
    flen[0] = lens[who[0]]
    src, dst = place[who].copy(), place[parents:].copy()
    if forks > 4:
        src[1], dst[2], flen[3] = -1, rows, -5      # skipped, skipped, no tokens
        dst[4] = src[4]                             # onto itself: skipped
    shares = g.integers(0, 4, pool)
    t, s = ints(table), ints(shares)
    want = oracle_pages.fork(src, dst, flen, table, block, shares, free)
    out = gpu_lib.gdn_paged_fork(ints(src), ints(dst), ints(flen), t, block, s, ints(free))
    same((t, s, *out), want, "fork")


def test_fork_of_nothing(gpu_lib):
    t, s, none = ints([[3, -1]]), ints(np.zeros(8)), ints(np.zeros(0))
    out = gpu_lib.gdn_paged_fork(none, none, none, t, 16, s, none)
    assert out[0].numel() == 0 and out[2].cpu().tolist() == [0, 0]
    assert t.cpu().tolist() == [[3, -1]]


# the last ones leave the form of one workgroup by their entries, by their pool, by both
@pytest.mark.parametrize("rows,ends,block,hi,pool,cut", [
    (4, 1, 16, 90, 64, None), (30, 30, 8, 300, 2000, None), (30, 11, 8, 300, 2000, 17),
    (6, 3, 64, 5000, 70001, None), (400, 300, 8, 700, 40000, None), (500, 77, 4, 500, 66000, 1000),
    (6, 3, 64, 5000, 32768, None), (6, 3, 64, 5000, 32769, None), (3, 2, 16, 8000, 9000, None),
])
def test_free(gpu_lib, rows, ends, block, hi, pool, cut):
    say("free", rows, ends, block, hi, pool)
    table, lens, shares, _ = shared_table(rows + ends, rows, hi, block, pool)
    g = np.random.default_rng(ends)
    who = g.permutation(rows)[:ends]
    wlen = lens[who].copy()
    if ends > 5:
        who[1], who[2], wlen[2] = -3, who[3], wlen[3]  # none, a row listed twice
        wlen[4] = 10 ** 6                              # longer than the row: the rest is null
    most = cut or min(ends * table.shape[1], pool)
    t, s = ints(table), ints(shares)
    want = oracle_pages.free(who, wlen, table, block, shares, most)
    freed, counts = gpu_lib.gdn_paged_free(ints(who), ints(wlen), t, block, s, max_freed=cut)
    same((t, s, freed, counts), want, "free")
    # the same rows again: nothing is left of them
    freed, counts = gpu_lib.gdn_paged_free(ints(who), ints(wlen), t, block, s, max_freed=cut)
    assert counts.item() == 0 and bool((freed == -1).all())
    same((t, s), want, "free again")


def test_free_into_the_rest_of_a_free_list(gpu_lib):
    table, lens, shares, free = shared_table(5, 8, 200, 16, 400)
    longer = ints(free[:5] + [99] * 300)
    t, s = ints(table), ints(shares)
    want = oracle_pages.free([2, 3], lens[2:4], table, 16, shares, 299)
    freed, counts = gpu_lib.gdn_paged_free(ints([2, 3]), ints(lens[2:4]), t, 16, s,
                                           freed=longer[5:304])
    same((t, s, freed, counts), want, "free")
    assert longer[:5].cpu().tolist() == free[:5] and longer[304].item() == 99


@pytest.mark.parametrize("rows,block,hi,pool,cut", [
    (1, 16, 0, 33, None), (1, 16, 500, 33, None), (12, 8, 200, 700, None), (12, 8, 200, 700, 5),
    (12, 8, 200, 700, 0), (7, 16, 900, 32768, None), (7, 16, 900, 32769, None),
    (200, 8, 700, 30000, None), (300, 4, 300, 100000, 50), (40, 64, 9000, 40000, None),
])
def test_compact(gpu_lib, rows, block, hi, pool, cut):
    say("compact", rows, block, hi, pool, cut)
    table, lens, shares, _ = shared_table(rows * 3 + hi, rows, hi, block, pool)
    table[:, -1] = 1  # behind the lengths: not held
    if rows > 5:
        table[2, 0], table[3, 0] = -1, pool + 7
    t, s = ints(table), ints(shares)
    most = pool // 2 if cut is None else cut
    want = oracle_pages.compact(lens, table, block, shares, most)
    out = gpu_lib.gdn_paged_compact(ints(lens), t, block, s, max_copies=cut)
    same((t, s, *out), want, "compact")
    if cut:  # the rest by further calls
        for _ in range(-(-int(want[4][1]) // cut)):
            table, shares = want[0], want[1]
            want = oracle_pages.compact(lens, table, block, shares, most)
            out = gpu_lib.gdn_paged_compact(ints(lens), t, block, s, max_copies=cut)
            same((t, s, *out), want, "compact on")
        assert want[4][1] == 0


def test_compact_of_a_full_and_of_an_empty_pool(gpu_lib):
    for table in ([[2, 0], [1, 3]], [[-1, -1], [-1, -1]]):
        t, s = ints(table), ints([0, 1, 0, 2])
        src, dst, counts = gpu_lib.gdn_paged_compact(ints([20, 32]), t, 16, s)
        assert counts.cpu().tolist() == [4 if table[0][0] >= 0 else 0, 0]
        assert t.cpu().tolist() == table and s.cpu().tolist() == [0, 1, 0, 2]
        assert bool((src == -1).all()) and bool((dst == -1).all())


# key/value caches, latent caches, state pools; pages of 16 bytes up to many pieces
@pytest.mark.parametrize("n_caches,shape,dtype,pairs", [
    (1, (8,), torch.bfloat16, 1), (2, (4, 24, 64), torch.bfloat16, 30), (7, (5, 3, 64), torch.float32, 9),
    (128, (16,), torch.float32, 50), (1, (64, 576), torch.bfloat16, 3), (3, (4, 128, 128), torch.float32, 6),
])
def test_copy(gpu_lib, n_caches, shape, dtype, pairs):
    say("copy", n_caches, shape, pairs)
    g = gen(pairs)
    n_blocks = 2 * pairs + 5
    caches = [torch.randn(n_blocks, *shape, generator=g).to(dtype) for _ in range(n_caches)]
    ids = torch.randperm(n_blocks, generator=g)
    src, dst = ids[:pairs].clone(), ids[pairs:2 * pairs].clone()
    if pairs > 4:
        src[1], dst[2], src[3] = -1, -1, n_blocks
        src[4] = src[0]  # one page to two places
    for count in (None, pairs // 2, pairs + 3, -1):
        used = pairs if count is None else max(min(count, pairs), 0)
        dev = [c.to(DEV) for c in caches]
        gpu_lib.gdn_paged_copy(dev, ints(src), ints(dst),
                               count=None if count is None else ints([count]))
        for c, d in zip(caches, dev):
            want = c.clone()
            for a, b in zip(src[:used].tolist(), dst[:used].tolist()):
                if 0 <= a < n_blocks and 0 <= b < n_blocks:
                    want[b] = c[a]
            assert torch.equal(want, d.cpu())


def test_copy_refuses(gpu_lib):
    a = torch.zeros(4, 8, dtype=torch.bfloat16, device=DEV)
    pair = ints([0]), ints([1])
    gpu_lib.gdn_paged_copy([], *pair)
    for caches in ([a, a[:2]], [a, torch.zeros(4, 16, device=DEV)], [a[:, :4]], [a, a.cpu()]):
        with pytest.raises(ValueError):
            gpu_lib.gdn_paged_copy(caches, *pair)
    with pytest.raises(gpu_lib.GdnError):
        gpu_lib.gdn_paged_copy([a] * 129, *pair)
    with pytest.raises(ValueError):
        gpu_lib.gdn_paged_copy([a], ints([0]).cpu(), ints([1]))
    with pytest.raises(ValueError):
        gpu_lib.gdn_paged_copy([a], ints([0]), ints([1, 2]))
