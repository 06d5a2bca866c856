"""gdn_paged_prefill against the fp64 oracle: head groups, lengths from one token on, pages that
end inside a step, prefixes, null pages, padded batches."""
import numpy as np
import pytest
import torch

from attn_util import assert_within, gen, normal, pages, tolerance
from gpu_util import DEV, say
from oracle import pages as oracle_pages

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def make(seed, lens, new, H, kv, d, block, dtype, null=False, pad=0):
    g = gen(seed)
    table, n_blocks = pages(g, lens, block)
    k, v = (normal(g, n_blocks, kv, block, d, dtype=dtype) for _ in range(2))
    used = torch.zeros(n_blocks, block, dtype=torch.bool)
    for i, n in enumerate(lens):
        for j in range(max(n, 0)):
            used[table[i, j // block], j % block] = True
    if null:  # pages that do not exist, before and among those that do
        table[0, 0] = -1
        table[-1, min(2, table.shape[1] - 1)] = n_blocks
    for c in (k, v):  # rows that nobody holds may hold anything
        c.transpose(1, 2)[~used] = float("nan")
    T = sum(new)
    q = normal(g, T + pad, H, d, dtype=dtype, scale=2.0)
    cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
    return q, k, v, table, cu, torch.tensor(lens, dtype=torch.int32)


def check(lib, args, scale, what, pad=0):
    q, k, v, table, cu, lens = args
    T = int(cu[-1])
    dev = [x.to(DEV) for x in args]
    o = torch.full_like(dev[0], 7.0)
    lib.gdn_paged_prefill(*dev, scale=scale, o=o)
    want, mag, top = oracle_pages.prefill(q[:T], torch.nan_to_num(k.float()),
                                          torch.nan_to_num(v.float()), table, cu, lens, scale)
    tol = tolerance(want, mag, top, q.shape[2], max(int(lens.max()), 1), q.dtype)
    assert_within(o[:T], want, tol, what)
    assert bool((o[T:] == 7.0).all()), "rows behind the last request"
    return dev, o


# (lens, new, H, kv, block): one token, odd sizes, several steps, several query tiles, a prefix of
# almost all, one request of no tokens between others, more groups than rows, one head
SHAPES = [
    ([1], [1], 4, 2, 16), ([5, 64, 65], [5, 64, 65], 8, 4, 24), ([300], [300], 8, 1, 64),
    ([700, 3, 0, 129], [40, 3, 0, 129], 6, 2, 20), ([257, 1000], [257, 1], 1, 1, 16),
    ([150, 90], [150, 20], 32, 2, 1), ([40, 500], [33, 64], 7, 7, 640), ([200], [17], 128, 1, 8),
]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_prefill(gpu_lib, shape, dtype, d):
    lens, new, H, kv, block = SHAPES[shape]
    say("prefill", lens, new, H, kv, block, dtype, d)
    check(gpu_lib, make(shape, lens, new, H, kv, d, block, dtype), d ** -0.5, "prefill")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_null_pages_and_padding(gpu_lib, dtype):
    check(gpu_lib, make(3, [100, 70, 90], [100, 5, 90], 8, 2, 128, 16, dtype, null=True, pad=9),
          128 ** -0.5, "null pages")
    # a request of which no page exists gives zeros
    args = make(4, [50, 40], [50, 40], 4, 4, 64, 16, dtype)
    args[3][1] = -1
    _, o = check(gpu_lib, args, 0.125, "no pages")
    assert bool((o[50:] == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [0.0, -0.09, 3.0])
def test_scales(gpu_lib, dtype, scale):
    check(gpu_lib, make(5, [130, 20], [90, 20], 4, 2, 64, 24, dtype), scale, f"scale {scale}")


def test_shorter_than_its_new_tokens(gpu_lib):
    """Lengths below the number of new tokens: the first ones see nothing, and give zeros."""
    args = make(6, [30, 80], [30, 80], 8, 4, 64, 16, BF16)
    args[5][0] = 12
    _, o = check(gpu_lib, args, 0.125, "short")
    assert bool((o[:18] == 0).all())


def test_longer_than_the_table(gpu_lib):
    """Tokens behind the last table column do not exist; positions stay."""
    q, k, v, table, cu, lens = make(7, [200], [60], 4, 2, 64, 16, F32)
    table = table[:, :9].contiguous()
    check(gpu_lib, (q, k, v, table, cu, lens), 0.125, "cut table")


def test_rows_behind_total_tokens(gpu_lib):
    """cu_seqlens beyond the rows that there are: the others keep their positions."""
    q, k, v, table, cu, lens = make(8, [90, 50], [90, 50], 4, 2, 64, 16, BF16)
    whole = gpu_lib.gdn_paged_prefill(*(x.to(DEV) for x in (q, k, v, table, cu, lens)), scale=0.125)
    for T in (120, 90, 41):
        got = gpu_lib.gdn_paged_prefill(*(x.to(DEV) for x in (q[:T].contiguous(), k, v, table, cu,
                                                              lens)), scale=0.125)
        assert_within(got, whole[:T].double().cpu().numpy(),
                      2.0 ** -7 * np.abs(whole[:T].double().cpu().numpy()) + 2.0 ** -7, "cut")


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 64), (BF16, 256)])
def test_many_steps_cut_between_workers(gpu_lib, dtype, d):
    """Long enough that every worker has a run of steps and most units are cut."""
    lens, new = [4000, 2500, 900], [300, 5, 900]
    check(gpu_lib, make(9, lens, new, 8, 2, d, 48, dtype), d ** -0.5, "long")


def test_a_score_that_outgrows_the_others(gpu_lib):
    """Keys that grow along the sequence: the reference of the exponents moves many times."""
    q, k, v, table, cu, lens = make(10, [900], [200], 4, 1, 64, 32, BF16)
    for j in range(900):
        k[table[0, j // 32], :, j % 32] *= 1 + j / 90
    check(gpu_lib, (q, k, v, table, cu, lens), 0.125, "growing keys")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_later_keys_of_any_value_have_no_weight(gpu_lib, dtype):
    """Infinite and NaN keys of later tokens, and values of 95 tokens on, reach no earlier row."""
    args = make(11, [400], [400], 8, 2, 64, 16, dtype)
    want = gpu_lib.gdn_paged_prefill(*(x.to(DEV) for x in args), scale=0.125)
    q, k, v, table, cu, lens = args
    for j, bad in ((300, float("nan")), (310, float("inf")), (390, -float("inf"))):
        k[table[0, j // 16], :, j % 16] = bad
        v[table[0, j // 16], :, j % 16] = bad
    got = gpu_lib.gdn_paged_prefill(*(x.to(DEV) for x in args), scale=0.125)
    assert torch.equal(got[:206], want[:206])
    k2 = make(11, [400], [400], 8, 2, 64, 16, dtype)
    k2[1].copy_(k)
    got = gpu_lib.gdn_paged_prefill(*(x.to(DEV) for x in k2), scale=0.125)
    assert torch.equal(got[:300], want[:300])


def test_the_same_from_run_to_run_and_for_any_page_order(gpu_lib):
    lens, new, H, kv, d, block = [1300, 700], [400, 650], 8, 2, 128, 16
    q, k, v, table, cu, l = make(12, lens, new, H, kv, d, block, BF16)
    one = gpu_lib.gdn_paged_prefill(*(x.to(DEV) for x in (q, k, v, table, cu, l)), scale=0.1)
    again = gpu_lib.gdn_paged_prefill(*(x.to(DEV) for x in (q, k, v, table, cu, l)), scale=0.1)
    perm = torch.randperm(k.shape[0], generator=gen(1))
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    k2[perm], v2[perm] = k, v
    t2 = torch.where(table >= 0, perm[table.clamp_min(0).long()].to(torch.int32), table)
    other = gpu_lib.gdn_paged_prefill(*(x.to(DEV) for x in (q, k2, v2, t2, cu, l)), scale=0.1)
    assert torch.equal(one, again) and torch.equal(one, other)


def test_one_token_each_is_a_decode_step(gpu_lib):
    lens = [1, 70, 333, 64]
    args = make(13, lens, [1] * 4, 8, 2, 128, 24, BF16)
    dev, o = check(gpu_lib, args, 128 ** -0.5, "single tokens")
    q, k, v, table, cu, l = dev
    step = gpu_lib.gdn_paged_decode(q, k, v, table, l, scale=128 ** -0.5)
    want, mag, top = oracle_pages.prefill(args[0], torch.nan_to_num(args[1].float()),
                                          torch.nan_to_num(args[2].float()), *args[3:], 128 ** -0.5)
    tol = tolerance(want, mag, top, 128, 333, BF16)
    assert_within(step, want, tol, "decode")


def test_no_rows_are_no_ops(gpu_lib):
    q, k, v, table, cu, lens = (x.to(DEV) for x in make(14, [20], [20], 4, 2, 64, 16, F32))
    out = gpu_lib.gdn_paged_prefill(q[:0], k, v, table, cu * 0, lens)
    assert out.shape == (0, 4, 64)
    out = gpu_lib.gdn_paged_prefill(q, k, v, table[:0], cu[:1], lens[:0], o=torch.full_like(q, 3.0))
    assert bool((out == 3.0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_more_requests_than_are_kept_near(gpu_lib, dtype):
    """2500 requests of 1 to 3 tokens, some of none: more bounds than the tables keep in LDS, more
    tiles than one pass of their kernel."""
    new = [(i * 7) % 4 for i in range(2500)]
    lens = [w + i % 9 if w else 0 for i, w in enumerate(new)]
    check(gpu_lib, make(15, lens, new, 2, 1, 64, 4, dtype), 0.125, "many requests")
