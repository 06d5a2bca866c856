"""Captured steps of shared pages replayed for other lengths: lengths, bounds, groups, tables and
lists are read on the device when a graph is replayed, so one recorded step serves every batch of
its sizes. Each replay against eager calls on the same inputs."""
import pytest
import torch

from attn_util import gen, normal
from gpu_util import DEV, say
from test_gpu_shared_run import ints

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32

B, WIDTH, BLOCK, POOL, T = 6, 200, 16, 1400, 500


def table(g, groups):
    """Rows of WIDTH pages; the rows of a group hold the first one's first 150 pages."""
    t = torch.randperm(POOL, generator=g)[:B * WIDTH].view(B, WIDTH).to(torch.int32)
    for a, z in groups:
        t[a + 1:z, :150] = t[a, :150]
    return t


# requests' lengths, group bounds, prefixes: long and short ones, groups elsewhere, requests that
# ended, nothing shared
BATCHES = [
    ([2500, 2410, 2433, 700, 650, 33], [0, 3, 5], [2400, 608], [(0, 3), (3, 5)]),
    ([90, 33, 1, 5, 2600, 3199], [0, 2, 3], [32, 0], [(0, 2)]),
    ([0, 2400, 0, 2415, 2420, 7], [0, 5, 5], [2400, 16], [(0, 5)]),
    ([1, 1, 1, 1, 1, 1], [6, 6, 6], [0, 0], []),
    ([0] * 6, [0, 3, 6], [16, 16], [(0, 3), (3, 6)]),
    ([2405, 2401, 2402, 2403, 2404, 2400], [0, 6, 6], [2400, 0], [(0, 6)]),
]


@pytest.mark.parametrize("least", [0, -1])
@pytest.mark.parametrize("dtype,d,P", [(BF16, 128, 1), (F32, 64, 2), (BF16, 256, 3)])
def test_shared_decode(gpu_lib, dtype, d, P, least):
    H, kv = 8, 2
    g = gen(5)
    kc, vc = (normal(g, POOL, kv, BLOCK, d, dtype=dtype).to(DEV) for _ in range(2))

    def batch(i):
        lens, cu, prefix, groups = BATCHES[i]
        h = gen(10 + i)
        return [normal(h, B, P, H, d, dtype=dtype, scale=2.0).to(DEV), table(h, groups).to(DEV),
                ints(lens), ints(cu), ints(prefix)]

    def call(x):
        return gpu_lib.gdn_paged_shared_decode(x[0], kc, vc, *x[1:], scale=d ** -0.5,
                                               min_bytes=least)
    replay(call, [batch(i) for i in range(len(BATCHES))], ("decode", dtype, d, P, least))


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 128), (F32, 64), (BF16, 256)])
def test_prompts(gpu_lib, dtype, d):
    """New tokens of all kinds of turns within 500 rows; rows behind the last are left alone."""
    H, kv = 8, 4
    g = gen(6)
    kc, vc = (normal(g, POOL, kv, BLOCK, d, dtype=dtype).to(DEV) for _ in range(2))
    turns = [([400, 0, 3, 90, 1, 6], [3000, 0, 3, 2000, 700, 6]), ([1] * B, [3199, 1, 64, 65, 2, 900]),
             ([0] * B, [5] * B), ([0, 0, 0, 0, 0, T], [0, 0, 0, 0, 0, T]),
             ([100, 100, 100, 100, 50, 50], [2900, 100, 40, 3000, 50, 1000]),
             ([T, 0, 9, 0, 0, 0], [3000, 7, 9, 0, 0, 0])]  # more than there are rows for

    def batch(i):
        new, lens = turns[i]
        h = gen(30 + i)
        cu = [0]
        for w in new:
            cu.append(cu[-1] + w)
        return [normal(h, T, H, d, dtype=dtype, scale=2.0).to(DEV), table(h, []).to(DEV), ints(cu),
                ints(lens), torch.full((T, H, d), 7.0, dtype=dtype, device=DEV)]

    def call(x):
        return gpu_lib.gdn_paged_prefill(x[0], kc, vc, *x[1:4], scale=d ** -0.5, o=x[4])
    replay(call, [batch(i) for i in range(len(turns))], ("prompts", dtype, d))


def replay(call, batches, what):
    """call(inputs) captured on the first batch, replayed for all in turn and back; every output,
    and every input that a call updates, as in an eager call."""
    say(*what)
    call([x.clone() for x in batches[0]])
    torch.cuda.synchronize()
    fixed = [x.clone() for x in batches[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call(fixed)
    outs = outs if isinstance(outs, (list, tuple)) else [outs]
    for turn, b in enumerate(batches + batches[::-1]):
        for f, x in zip(fixed, b):
            f.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in [*outs, *fixed]]
        now = [x.clone() for x in b]
        want = call(now)
        want = [*(want if isinstance(want, (list, tuple)) else [want]), *now]
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(got, want)):
            assert torch.equal(x, y), f"{what} replay {turn}: tensor {i}"


@pytest.mark.parametrize("rows,pool", [(12, 400), (200, 60000)])  # one workgroup, and several
def test_forks_ends_and_compactions(gpu_lib, rows, pool):
    """Other forks, ends and live pages in every replay."""
    width, block = 40, 8

    def batch(i):
        g = gen(50 + i)
        t = torch.full((rows, width), -1, dtype=torch.int32)
        held = torch.randint(1, width, (rows // 2,), generator=g)
        ids = torch.randperm(pool, generator=g).to(torch.int32)
        at = 0
        for r, n in enumerate(held.tolist()):
            t[r, :n] = ids[at:at + n]
            at += n
        n = 4
        src = torch.randint(rows // 2, (n,), generator=g)
        lens = torch.zeros(rows, dtype=torch.long)
        lens[:rows // 2] = held * block - torch.randint(block, (rows // 2,), generator=g)
        dst = rows // 2 + torch.randperm(rows // 2, generator=g)[:n]
        fork = (lens[src] * torch.rand(n, generator=g)).long()
        if i == 2:
            src[0], fork[1], dst[2] = -1, 0, rows + 5      # some that are none
        after = lens.clone()
        ok = (src >= 0) & (dst < rows)
        after[dst[ok]] = fork[ok]
        gone = torch.randperm(rows // 2, generator=g)[:3]
        gone_lens = lens[gone].clone()
        after[gone] = 0
        return [x.to(torch.int32).to(DEV) for x in (
            src, dst, fork, t, torch.zeros(pool), ids[at:at + 50], gone, gone_lens, after)]

    def call(x):
        src, dst, fork, t, shares, free, gone, gone_lens, after = x
        a = gpu_lib.gdn_paged_fork(src, dst, fork, t, block, shares, free)
        b = gpu_lib.gdn_paged_free(gone, gone_lens, t, block, shares)
        c = gpu_lib.gdn_paged_compact(after, t, block, shares)
        return [*a, *b, *c]
    replay(call, [batch(i) for i in range(5)], ("pages", rows, pool))
