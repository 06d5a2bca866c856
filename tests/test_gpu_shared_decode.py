"""gdn_paged_shared_decode against the fp64 oracle, and against gdn_paged_decode: groups of all
sizes, prefixes of any length, requests outside groups, padded rows."""
import numpy as np
import pytest
import torch

from attn_util import assert_within, gen, normal, tolerance
from gpu_util import DEV, say
from oracle import pages as oracle_pages

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def make(seed, sizes, prefix, own, P, H, kv, d, block, dtype, before=0, part=True):
    """Groups of these sizes and prefix lengths; own[b] tokens of request b behind its prefix;
    `before` requests come before the first group, the rest of `own` behind the last. With `part`
    the whole prefix is named as shared though its last page is not whole: that page is shared by
    the rows only where nothing follows it."""
    g = gen(seed)
    B = len(own)
    cu = [before]
    for s in sizes:
        cu.append(cu[-1] + s)
    skip = [0] * B
    for i, x in enumerate(prefix):
        for b in range(cu[i], cu[i + 1]):
            skip[b] = x if part else x // block * block
    lens = [skip[b] + own[b] if skip[b] else own[b] for b in range(B)]
    need = [-(-x // block) for x in lens]
    most = sum(need) + sum(-(-x // block) for x in prefix) + 5
    ids = torch.randperm(most, generator=g).tolist()
    table = torch.full((B, max(need + [1]) + 2), -1, dtype=torch.int32)
    k, v = (normal(g, most, kv, block, d, dtype=dtype) for _ in range(2))
    at = 0
    for b in range(B):
        first = next((cu[i] for i in range(len(sizes)) if cu[i] <= b < cu[i + 1]), b)
        whole = skip[b] // block if b > first else 0
        table[b, :whole] = table[first, :whole]
        for p in range(whole, need[b]):
            table[b, p] = ids[at]
            at += 1
        if b > first and skip[b] % block:  # the same tokens in a page of its own
            p, n = skip[b] // block, skip[b] % block
            for c in (k, v):
                c[table[b, p], :, :n] = c[table[first, p], :, :n]
    used = torch.zeros(most, block, dtype=torch.bool)
    for b in range(B):
        for j in range(lens[b]):
            used[table[b, j // block], j % block] = True
    for c in (k, v):
        c.transpose(1, 2)[~used] = float("nan")
    q = normal(g, B, P, H, d, dtype=dtype, scale=2.0)
    named = [x if part else x // block * block for x in prefix]
    return (q, k, v, table, torch.tensor(lens, dtype=torch.int32),
            torch.tensor(cu, dtype=torch.int32), torch.tensor(named, dtype=torch.int32))


def check(lib, args, scale, what):
    q, k, v, table, lens, cu, prefix = args
    dev = [x.to(DEV) for x in args]
    o = lib.gdn_paged_shared_decode(*dev, scale=scale, min_bytes=0)  # (apart, however little)
    want, mag, top = oracle_pages.shared_decode(q, torch.nan_to_num(k.float()),
                                                torch.nan_to_num(v.float()), table, lens, cu,
                                                prefix, scale)
    tol = tolerance(want, mag, top, q.shape[3], max(int(lens.max()), 1), q.dtype)
    assert_within(o, want, tol, what)
    return dev, o, want, tol


# (group sizes, prefix lengths, own tokens, before, P, H, kv, block)
CASES = [
    ([2], [16], [1, 1], 0, 1, 4, 2, 16),
    ([3, 2], [70, 130], [5, 1, 90, 33, 2], 0, 1, 8, 4, 24),
    ([5], [513], [3, 3, 3, 3, 200], 0, 3, 6, 2, 20),
    ([1, 4, 1], [100, 64, 50], [9, 9, 70, 8, 7, 6, 40, 300], 1, 2, 8, 1, 16),
    ([40], [300], list(range(1, 41)), 0, 1, 8, 1, 64),
    ([2, 0, 3], [40, 77, 0], [4, 5, 6, 7, 8, 9], 0, 1, 7, 7, 8),
    ([6, 6], [900, 31], [20] * 13, 0, 4, 32, 2, 32),
]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("part", [True, False])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_shared(gpu_lib, case, part, dtype, d):
    sizes, prefix, own, before, P, H, kv, block = CASES[case]
    say("shared", sizes, prefix, P, H, kv, block, dtype, d, part)
    own = [max(x, P) for x in own]
    args = make(case, sizes, prefix, own, P, H, kv, d, block, dtype, before, part)
    dev, o, want, tol = check(gpu_lib, args, d ** -0.5, "shared")
    plain = gpu_lib.gdn_paged_decode(*dev[:5], scale=d ** -0.5)
    assert_within(plain, want, tol, "plain decode of the same batch")
    rule = gpu_lib.gdn_paged_shared_decode(*dev, scale=d ** -0.5)  # too little to be spared
    assert_within(rule, want, tol, "each request its own prefix")
    assert torch.equal(rule, gpu_lib.gdn_paged_shared_decode(*dev, scale=d ** -0.5,
                                                             min_bytes=2 ** 62))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_long_prefix_over_all_workers(gpu_lib, dtype):
    args = make(21, [9], [5000], [1, 2, 3, 40, 500, 6, 7, 8, 9], 1, 8, 2, 128, 64, dtype)
    check(gpu_lib, args, 128 ** -0.5, "long prefix")


def test_long_own_keys(gpu_lib):
    args = make(22, [3], [130], [4000, 3, 2500], 2, 8, 2, 64, 16, BF16)
    check(gpu_lib, args, 0.125, "long own keys")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_short_and_padded_requests(gpu_lib, dtype):
    """Requests of a group that are shorter than its prefix, of no tokens, of fewer than P."""
    args = make(23, [6], [200], [5] * 7, 3, 8, 2, 64, 16, dtype)
    args[4][1], args[4][2], args[4][4], args[4][5] = 0, 2, 77, 200
    _, o, want, _ = check(gpu_lib, args, 0.125, "short")
    assert bool((o[1] == 0).all()) and bool((o[2, 0] == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_negative_lengths_count_as_none(gpu_lib, dtype):
    """Down to the smallest number there is, also where several positions come before it."""
    args = [x.to(DEV) for x in make(32, [4], [200], [5] * 5, 4, 8, 2, 64, 16, dtype)]
    args[4][1], args[4][2] = 0, 0
    want = gpu_lib.gdn_paged_shared_decode(*args, scale=0.125, min_bytes=0)
    args[4][1], args[4][2] = -2 ** 31, -3
    o = gpu_lib.gdn_paged_shared_decode(*args, scale=0.125, min_bytes=0)
    assert bool((o[1:3] == 0).all()) and torch.equal(o, want)


def test_null_pages(gpu_lib):
    args = make(24, [4], [128], [30] * 5, 1, 8, 4, 64, 16, BF16)
    args[3][:4, 2] = -1                        # of the prefix
    args[3][3, 8], args[3][4, 0] = 10 ** 6, -1  # of own keys
    check(gpu_lib, args, 0.125, "null pages")


@pytest.mark.parametrize("scale", [0.0, -0.1])
def test_scales(gpu_lib, scale):
    check(gpu_lib, make(25, [3], [90], [5, 6, 7], 1, 4, 2, 64, 16, BF16), scale, "scale")


def test_no_groups_is_a_decode_step(gpu_lib):
    args = make(26, [], [], [5, 100, 700], 1, 8, 2, 128, 16, BF16)
    dev, o, _, _ = check(gpu_lib, args, 0.1, "no groups")
    step = gpu_lib.gdn_paged_decode(*dev[:5], scale=0.1)
    assert torch.equal(o, step)
    one = gpu_lib.gdn_paged_shared_decode(dev[0][:, 0].contiguous(), *dev[1:], scale=0.1)
    assert torch.equal(one, o[:, 0])


def test_the_same_from_run_to_run(gpu_lib):
    args = [x.to(DEV) for x in make(27, [5, 4], [700, 333], [30] * 10, 2, 16, 2, 128, 32, BF16)]
    one = gpu_lib.gdn_paged_shared_decode(*args, scale=0.1, min_bytes=0)
    for _ in range(3):
        assert torch.equal(one, gpu_lib.gdn_paged_shared_decode(*args, scale=0.1, min_bytes=0))


def test_groups_that_break_the_contract_touch_nothing_else(gpu_lib):
    """Bounds that decrease, overlap or leave the batch: outputs of some kind, within the arrays."""
    args = [x.to(DEV) for x in make(28, [3, 3], [64, 64], [9] * 6, 1, 4, 2, 64, 16, F32)]
    for cu in ([0, 6, 3], [4, 2, 6], [-5, 3, 60], [0, 6, 6], [7, 8, 9]):
        args[5] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        o = gpu_lib.gdn_paged_shared_decode(*args, scale=0.1, min_bytes=0)
        assert o.shape == args[0].shape
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_the_rule_takes_prefixes_apart_where_much_is_spared(gpu_lib, dtype):
    """40 requests behind 2000 tokens, 2 heads of 256: 160 MB (320 in fp32)."""
    args = make(29, [40], [2000], list(range(1, 41)), 1, 4, 2, 256, 64, dtype)
    dev, o, want, tol = check(gpu_lib, args, 1 / 16, "apart")
    assert torch.equal(o, gpu_lib.gdn_paged_shared_decode(*dev, scale=1 / 16))


def test_the_rule_leaves_fp32_groups_of_few_rows_to_the_decode_kernel(gpu_lib):
    args = [x.to(DEV) for x in make(30, [3], [9000], [9, 9, 9], 1, 8, 8, 256, 64, F32)]
    rule = gpu_lib.gdn_paged_shared_decode(*args, scale=1 / 16)  # 295 MB spared, 3 rows
    assert torch.equal(rule, gpu_lib.gdn_paged_shared_decode(*args, scale=1 / 16, min_bytes=2 ** 62))
    # bf16 ones are taken apart
    half = [x.to(BF16) if x.dtype == F32 else x for x in args]
    apart = gpu_lib.gdn_paged_shared_decode(*half, scale=1 / 16)
    assert torch.equal(apart, gpu_lib.gdn_paged_shared_decode(*half, scale=1 / 16, min_bytes=0))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_more_groups_than_are_kept_near(gpu_lib, dtype):
    """2100 groups, and tables of more tiles than one pass of their kernel."""
    args = make(31, [2] * 2100, [5] * 2100, [1] * 4201, 1, 2, 1, 64, 4, dtype, part=False)
    check(gpu_lib, args, 0.125, "many groups")
