"""gdn_paged_plan, gdn_paged_append, gdn_latent_append and gdn_paged_decode on the GPU against
the fp64 reference."""
import numpy as np
import pytest
import torch

from attn_util import assert_within, gen, normal, pages, tolerance
from gated_delta_rule_prefill_amd import gdn
from gpu_util import DEV, say
from oracle import attention

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------------------------ plan
def _plan_case(seed, ctx, new, block, width=None, n_free=None, max_tokens=None):
    g = gen(seed)
    n = len(ctx)
    need = [-(-(max(c, 0) + max(w, 0)) // block) for c, w in zip(ctx, new)]
    held = [-(-max(c, 0) // block) for c in ctx]
    width = max(need + [1]) + 1 if width is None else width
    ids = torch.randperm(sum(need) + 10, generator=g).to(torch.int32)
    table = torch.full((n, width), -7, dtype=torch.int32)  # a value that must survive
    at = 0
    for i in range(n):
        k = min(held[i], width)
        table[i, :k] = ids[at:at + k]
        at += k
    free = ids[at:]
    if n_free is not None:
        free = free[:n_free]
    T = sum(max(w, 0) for w in new) if max_tokens is None else max_tokens
    return (torch.tensor(ctx, dtype=torch.int32), torch.tensor(new, dtype=torch.int32), table,
            free.clone(), block, T)


def _check_plan(case):
    ctx, new, table, free, block, T = case
    want = attention.plan(ctx.tolist(), new.tolist(), table, free, block, T)
    d = [t.to(DEV) for t in (ctx, new, table, free)]
    out = gdn.gdn_paged_plan(d[0], d[1], d[2], d[3], block, T)
    torch.cuda.synchronize()
    for name, got, ref in zip(("table", "cu", "lens", "slots", "positions", "counts"),
                              (d[2], *out), want):
        assert np.array_equal(got.cpu().numpy(), ref), name
    assert torch.equal(d[3].cpu(), free)


@pytest.mark.parametrize("ctx,new,block", [
    ([0], [1], 16), ([5], [0], 8), ([0, 0, 0], [0, 0, 0], 4), ([7, 8, 9], [1, 1, 1], 8),
    ([0, 3, 64, 100, 0], [1000, 0, 64, 1, 4097], 64), ([3, 0, 9], [5, 2, 30], 1),
    ([0, 17], [3000, 1500], 640), ([-3, 4], [5, -2], 3)])
def test_plan(ctx, new, block):
    say(f"case plan {ctx} {new} {block}")
    _check_plan(_plan_case(1, ctx, new, block))


@pytest.mark.parametrize("n", [1, 255, 256, 257, 700, 3001])
def test_plan_many_requests(n):
    say(f"case plan n={n}")
    g = gen(n)
    ctx = torch.randint(0, 200, (n,), generator=g).tolist()
    new = torch.randint(0, 9, (n,), generator=g).tolist()
    _check_plan(_plan_case(2, ctx, new, 16))


def test_plan_padded_buffers_and_short_free_list():
    say("case plan padded, short free list, narrow table, short buffers")
    ctx, new = [10, 0, 33], [20, 50, 1]
    _check_plan(_plan_case(3, ctx, new, 8, max_tokens=1111))
    _check_plan(_plan_case(4, ctx, new, 8, n_free=3))
    _check_plan(_plan_case(5, ctx, new, 8, n_free=0))
    _check_plan(_plan_case(6, ctx, new, 8, width=3))
    _check_plan(_plan_case(7, ctx, new, 8, max_tokens=37))
    _check_plan(_plan_case(8, ctx, new, 8, max_tokens=0))


def test_plan_without_requests():
    say("case plan n=0")
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    cu, lens, slots, pos, counts = gdn.gdn_paged_plan(
        e, e, torch.empty(0, 4, dtype=torch.int32, device=DEV), e, 16, 10)
    torch.cuda.synchronize()
    assert cu.tolist() == [0] and counts.tolist() == [0, 0]
    assert slots.tolist() == [-1] * 10 and pos.tolist() == [0] * 10


def test_plan_keeps_null_entries():
    """A null entry among the held pages gives its tokens no slot."""
    say("case plan null entry")
    case = list(_plan_case(9, [12, 5], [6, 2], 8))
    case[2][0, 1] = -1
    _check_plan(tuple(case))


# ---------------------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype,d,heads,block,T", [
    (BF16, 64, 1, 16, 1), (BF16, 128, 3, 7, 50), (BF16, 256, 2, 64, 333), (F32, 64, 5, 16, 129),
    (F32, 256, 1, 1, 17)])
def test_paged_append(dtype, d, heads, block, T):
    say(f"case append {dtype} d={d} heads={heads} block={block} T={T}")
    g = gen(T)
    n_blocks = -(-T // block) + 2
    qkv = normal(g, T, 3 * heads, d, dtype=dtype)
    kc, vc = (normal(g, n_blocks, heads, block, d, dtype=dtype) for _ in range(2))
    slots = torch.randperm(n_blocks * block, generator=g)[:T]
    if T > 3:
        slots[1], slots[2] = -1, n_blocks * block  # skipped tokens
    want = []
    for src, cache in ((qkv[:, heads:2 * heads], kc), (qkv[:, 2 * heads:], vc)):
        w = cache.clone()
        for t, s in enumerate(slots.tolist()):
            if 0 <= s < n_blocks * block:
                w[s // block, :, s % block] = src[t]
        want.append(w)
    dq, dk, dv, ds = (x.to(DEV) for x in (qkv, kc, vc, slots))
    gdn.gdn_paged_append(dq[:, heads:2 * heads], dq[:, 2 * heads:], ds, dk, dv)
    torch.cuda.synchronize()
    assert torch.equal(dk.cpu(), want[0]) and torch.equal(dv.cpu(), want[1])


@pytest.mark.parametrize("dtype,rank,rope,block,T", [
    (BF16, 512, 64, 64, 200), (BF16, 256, 64, 5, 1), (F32, 256, 64, 16, 77), (BF16, 24, 8, 3, 40)])
def test_latent_append(dtype, rank, rope, block, T):
    say(f"case latent append {dtype} {rank} {rope} {block} {T}")
    g = gen(T)
    n_blocks = -(-T // block) + 2
    kv = normal(g, T, rank + rope + 8, dtype=dtype)
    cache = normal(g, n_blocks, block, rank + rope, dtype=dtype)
    slots = torch.randperm(n_blocks * block, generator=g)[:T]
    if T > 3:
        slots[0], slots[3] = -5, n_blocks * block + 1
    want = cache.clone().view(-1, rank + rope)
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < n_blocks * block:
            want[s] = kv[t, :rank + rope]
    dkv, dc, ds = (x.to(DEV) for x in (kv, cache, slots))
    gdn.gdn_latent_append(dkv[:, :rank], dkv[:, rank:rank + rope], ds, dc)
    torch.cuda.synchronize()
    assert torch.equal(dc.cpu().view(-1, rank + rope), want)


def test_append_of_no_tokens_changes_nothing():
    say("case append T=0")
    kc = torch.ones(2, 1, 4, 64, dtype=BF16, device=DEV)
    e = torch.empty(0, 1, 64, dtype=BF16, device=DEV)
    gdn.gdn_paged_append(e, e, torch.empty(0, dtype=torch.int64, device=DEV), kc, kc.clone())
    torch.cuda.synchronize()
    assert torch.equal(kc, torch.ones_like(kc))


# ---------------------------------------------------------------------------------- decode
def _decode_case(seed, lens, P, H, kv, d, block, dtype, poison=True, q_scale=2.0):
    g = gen(seed)
    table, n_blocks = pages(g, lens, block)
    kc = normal(g, n_blocks, kv, block, d, dtype=dtype)
    vc = normal(g, n_blocks, kv, block, d, dtype=dtype)
    if poison:  # what no request has: unused pages and the rows behind each request's last
        used = torch.zeros(n_blocks, block, dtype=torch.bool)
        for i, x in enumerate(lens):
            for j in range(max(x, 0)):
                used[int(table[i, j // block]), j % block] = True
        hole = (~used)[:, None, :, None].expand_as(kc)
        kc = torch.where(hole, torch.tensor(float("nan"), dtype=dtype), kc)
        vc = torch.where(hole, torch.tensor(float("inf"), dtype=dtype), vc)
    q = normal(g, len(lens), P, H, d, dtype=dtype, scale=q_scale)
    return q, kc, vc, table, torch.tensor(lens, dtype=torch.int32), d ** -0.5


def _run_decode(case, **kw):
    q, kc, vc, table, lens, scale = case
    o = gdn.gdn_paged_decode(*(x.to(DEV) for x in (q, kc, vc, table, lens)), scale=scale, **kw)
    torch.cuda.synchronize()
    return o


def _check_decode(case):
    q, kc, vc, table, lens, scale = case
    clean = [torch.nan_to_num(x.float(), nan=0.0, posinf=0.0).double() for x in (kc, vc)]
    want, mag, top = attention.paged_decode(q, *clean, table, lens, scale)
    o = _run_decode(case)
    n = int(lens.max().clamp_min(0))
    assert_within(o, want, tolerance(want, mag, top, q.shape[3], n, q.dtype))
    return o


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H,kv,P,block", [(1, 1, 1, 16), (8, 2, 1, 64), (6, 2, 3, 24),
                                          (16, 1, 2, 5), (7, 1, 5, 640)])
def test_paged_decode(dtype, d, H, kv, P, block):
    say(f"case decode {dtype} d={d} H={H} kv={kv} P={P} block={block}")
    _check_decode(_decode_case(d + H, [1, 130, 0, 17, 300, 64, 2], P, H, kv, d, block, dtype))


@pytest.mark.parametrize("H,kv,P", [(64, 1, 1), (64, 1, 2), (40, 2, 16), (128, 1, 1)])
@pytest.mark.parametrize("d", [64, 256])
def test_paged_decode_many_rows(H, kv, P, d):
    """More query rows than one tile."""
    say(f"case decode rows H={H} kv={kv} P={P} d={d}")
    _check_decode(_decode_case(3, [90, 5, 257], P, H, kv, d, 32, BF16))


@pytest.mark.parametrize("lens", [[1], [31], [32], [33], [127], [128], [129], [5000], [20011]])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_paged_decode_lengths(lens, dtype):
    """One request, from one token to a length that every workgroup takes a part of."""
    say(f"case decode length {lens} {dtype}")
    _check_decode(_decode_case(lens[0], lens, 1, 4, 2, 64, 64, dtype))


def test_paged_decode_ragged_batch():
    say("case decode ragged")
    g = gen(5)
    lens = torch.randint(0, 400, (301,), generator=g).tolist()
    lens[7], lens[100] = 6000, 0
    _check_decode(_decode_case(6, lens, 1, 4, 1, 128, 16, BF16))


def test_paged_decode_positions_before_the_start():
    """A verify step of more positions than the request has tokens: the first see none."""
    say("case decode P > len")
    case = _decode_case(8, [2, 0, 5, 1], 4, 4, 2, 64, 8, BF16)
    o = _check_decode(case)
    assert torch.equal(o[0, :2], torch.zeros_like(o[0, :2]))
    assert torch.equal(o[1], torch.zeros_like(o[1]))


@pytest.mark.parametrize("block", [8, 64, 100])
def test_paged_decode_null_blocks(block):
    """Null entries, ids past the pool and a length past the table: those tokens do not exist."""
    say(f"case decode null {block}")
    whole = -(-700 // block) * block  # its length is raised below: every row of its pages counts
    case = list(_decode_case(9, [whole, 300, 250], 2, 4, 2, 128, block, BF16))
    case[3][0, 1] = -1
    case[3][0, 3] = 1 << 30
    case[3][1, :3] = -9
    case[3][2, :] = -1
    case[4][0] = 1 << 20
    _check_decode(tuple(case))


def test_paged_decode_extreme_scores():
    """Scores hundreds apart, all very negative, or all equal."""
    say("case decode extremes")
    for seed, scale in ((1, 300.0), (2, -300.0), (3, 0.0)):
        case = list(_decode_case(seed, [77, 500], 1, 4, 2, 64, 16, F32, q_scale=1.0))
        case[5] = scale / 8
        _check_decode(tuple(case))
    case = list(_decode_case(4, [77, 500], 1, 4, 2, 64, 16, BF16))
    case[1] = torch.full_like(case[1], -2.0)  # every score the same, far from zero
    case[0] = torch.full_like(case[0], 3.0)
    _check_decode(tuple(case))


def test_paged_decode_is_the_same_every_time_and_for_any_page_order():
    say("case decode determinism")
    lens = [4000, 33, 900]
    case = _decode_case(10, lens, 2, 8, 2, 128, 16, BF16, poison=False)
    q, kc, vc, table, ln, scale = case
    a, b = _run_decode(case), _run_decode(case)
    assert torch.equal(a, b)
    perm = torch.randperm(kc.shape[0], generator=gen(11))
    inv = torch.argsort(perm)
    moved = torch.where(table >= 0, inv[table.clamp_min(0).long()].to(torch.int32), table)
    assert torch.equal(_run_decode((q, kc[perm], vc[perm], moved, ln, scale)), a)


def test_paged_decode_three_and_four_dims_agree():
    say("case decode dims")
    q, kc, vc, table, ln, scale = _decode_case(12, [50, 60], 1, 4, 4, 64, 16, BF16)
    a = _run_decode((q, kc, vc, table, ln, scale))
    b = _run_decode((q[:, 0].contiguous(), kc, vc, table, ln, scale))
    assert b.shape == (2, 4, 64) and torch.equal(a[:, 0], b)
