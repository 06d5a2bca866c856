"""gdn_latent_decode (absorbed form) and gdn_latent_prefill (expanded form) on the GPU against
the fp64 reference, which evaluates each in its own form."""
import numpy as np
import pytest
import torch

from attn_util import assert_within, gen, normal, pages
from gated_delta_rule_prefill_amd import gdn
from gpu_util import DEV, say
from oracle import attention

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
ROPE = 64
# An output is a sum of many independent roundings: 7 standard deviations hold with a margin of
# 1e-6 over a million outputs even for heavier tails than a normal's.
SIGMAS = 7.0
HALF_STEP = 2.0 ** -8


def _cache(g, lens, block, R, poison):
    table, n_blocks = pages(g, lens, block)
    cache = normal(g, n_blocks, block, R + ROPE)
    if poison:  # what no request has: unused pages and the rows behind each request's last
        used = torch.zeros(n_blocks, block, dtype=torch.bool)
        for i, x in enumerate(lens):
            for j in range(max(x, 0)):
                used[int(table[i, j // block]), j % block] = True
        cache[~used] = float("nan")
    return table, cache


def _weights(g, H, R, d):
    return normal(g, H, 2 * d, R, scale=R ** -0.5)


def _tolerance(qn, qp, w, cache, table, limits, o, scale):
    """SIGMAS x attention.latent_error for packed rows qn [T, H, .]; limits[t] = (request, keys
    that the row sees)."""
    f = [x.double().numpy() for x in (qn, qp, w)]
    c = torch.nan_to_num(cache.float()).double().numpy()
    tol = np.zeros(o.shape)
    for t, (b, n) in enumerate(limits):
        pos, rows = attention._latent_rows(c, table[b].numpy(), n)
        for h in range(o.shape[1]):
            tol[t, h] = attention.latent_error(f[0][t, h], f[1][t, h], f[2][h], rows, o[t, h],
                                               scale, HALF_STEP)
    return SIGMAS * tol + 1e-30


# ---------------------------------------------------------------------------------- decode
def _decode_case(seed, lens, P, H, R, d, block, poison=True, q_scale=1.5):
    g = gen(seed)
    table, cache = _cache(g, lens, block, R, poison)
    B = len(lens)
    return (normal(g, B, P, H, d, scale=q_scale), normal(g, B, P, H, ROPE, scale=q_scale),
            _weights(g, H, R, d), cache, table, torch.tensor(lens, dtype=torch.int32),
            (d + ROPE) ** -0.5)


def _run_decode(case, **kw):
    o = gdn.gdn_latent_decode(*(x.to(DEV) for x in case[:6]), scale=case[6], **kw)
    torch.cuda.synchronize()
    return o


def _check_decode(case):
    qn, qp, w, cache, table, lens, scale = case
    B, P, H, d = qn.shape
    clean = torch.nan_to_num(cache.float()).double()
    want = attention.latent_absorbed(qn, qp, w, clean, table, lens, scale)
    o = _run_decode(case)
    limits = [(b, int(lens[b]) - P + p + 1) for b in range(B) for p in range(P)]
    flat = want.reshape(B * P, H, d)
    tol = _tolerance(qn.view(B * P, H, d), qp.view(B * P, H, ROPE), w, cache, table, limits, flat,
                     scale)
    assert_within(o.view(B * P, H, d), flat, tol)
    return o


@pytest.mark.parametrize("R,d", [(512, 128), (256, 64), (512, 64), (256, 128)])
@pytest.mark.parametrize("H,P,block", [(1, 1, 16), (16, 1, 64), (20, 1, 64), (6, 3, 24),
                                       (40, 1, 5), (16, 4, 640)])
def test_latent_decode(R, d, H, P, block):
    say(f"case latent decode R={R} d={d} H={H} P={P} block={block}")
    _check_decode(_decode_case(R + d + H, [1, 130, 0, 17, 300, 64, 2], P, H, R, d, block))


@pytest.mark.parametrize("H,P", [(128, 1), (70, 2)])
def test_latent_decode_many_rows(H, P):
    """More query rows than one row tile holds."""
    say(f"case latent decode rows H={H} P={P}")
    _check_decode(_decode_case(3, [90, 5, 257], P, H, 512, 128, 32))


@pytest.mark.parametrize("n", [1, 15, 16, 63, 64, 65, 5000, 17011])
def test_latent_decode_lengths(n):
    """One request, from one token to a length that every workgroup takes a part of."""
    say(f"case latent decode length {n}")
    _check_decode(_decode_case(n, [n], 1, 2, 512, 128, 64))


def test_latent_decode_ragged_batch():
    say("case latent decode ragged")
    g = gen(5)
    lens = torch.randint(0, 300, (70,), generator=g).tolist()
    lens[7], lens[20] = 4000, 0
    _check_decode(_decode_case(6, lens, 1, 4, 256, 64, 16))


def test_latent_decode_positions_before_the_start():
    say("case latent decode P > len")
    o = _check_decode(_decode_case(8, [2, 0, 5, 1], 4, 3, 512, 128, 8))
    assert torch.equal(o[0, :2], torch.zeros_like(o[0, :2]))
    assert torch.equal(o[1], torch.zeros_like(o[1]))


@pytest.mark.parametrize("block", [8, 64, 100])
def test_latent_decode_null_blocks(block):
    say(f"case latent decode null {block}")
    whole = -(-700 // block) * block
    case = list(_decode_case(9, [whole, 300, 250], 2, 4, 512, 128, block))
    case[4][0, 1] = -1
    case[4][0, 3] = 1 << 30
    case[4][1, :3] = -9
    case[4][2, :] = -1
    case[5][0] = 1 << 20
    _check_decode(tuple(case))


def test_latent_decode_is_the_same_every_time_and_for_any_page_order():
    say("case latent decode determinism")
    case = _decode_case(10, [4000, 33, 900], 2, 20, 512, 128, 16, poison=False)
    a, b = _run_decode(case), _run_decode(case)
    assert torch.equal(a, b)
    qn, qp, w, cache, table, ln, scale = case
    perm = torch.randperm(cache.shape[0], generator=gen(11))
    inv = torch.argsort(perm)
    moved = torch.where(table >= 0, inv[table.clamp_min(0).long()].to(torch.int32), table)
    assert torch.equal(_run_decode((qn, qp, w, cache[perm], moved, ln, scale)), a)


def test_latent_decode_three_and_four_dims_agree():
    say("case latent decode dims")
    case = _decode_case(12, [50, 60], 1, 4, 512, 128, 16)
    a = _run_decode(case)
    b = _run_decode((case[0][:, 0].contiguous(), case[1][:, 0].contiguous(), *case[2:]))
    assert b.shape == (2, 4, 128) and torch.equal(a[:, 0], b)


# --------------------------------------------------------------------------------- prefill
def _prefill_case(seed, ctx, new, H, R, d, block, poison=True, q_scale=1.5):
    g = gen(seed)
    lens = [c + w for c, w in zip(ctx, new)]
    table, cache = _cache(g, lens, block, R, poison)
    T = sum(new)
    cu = torch.tensor([0] + np.cumsum(new).tolist(), dtype=torch.int32)
    return (normal(g, T, H, d, scale=q_scale), normal(g, T, H, ROPE, scale=q_scale),
            _weights(g, H, R, d), cache, table, cu, torch.tensor(lens, dtype=torch.int32),
            (d + ROPE) ** -0.5)


def _run_prefill(case, keys=None, **kw):
    keys = int(case[6].clamp_min(0).sum()) if keys is None else keys
    o = gdn.gdn_latent_prefill(*(x.to(DEV) for x in case[:7]), keys, scale=case[7], **kw)
    torch.cuda.synchronize()
    return o


def _check_prefill(case, keys=None, every=1):
    """`every`: tokens of which the tolerance is worked out (it costs a pass over the keys)."""
    qn, qp, w, cache, table, cu, lens, scale = case
    clean = torch.nan_to_num(cache.float()).double()
    want = attention.latent_expanded(qn, qp, w, clean, table, cu, lens, scale)
    o = _run_prefill(case, keys)
    limits = []
    for i in range(len(lens)):
        new = int(cu[i + 1] - cu[i])
        limits += [(i, int(lens[i]) - new + t + 1) for t in range(new)]
    pick = list(range(0, len(limits), every))
    tol = _tolerance(qn[pick], qp[pick], w, cache, table, [limits[t] for t in pick], want[pick],
                     scale)
    assert_within(o[pick], want[pick], tol)
    assert torch.isfinite(o.float()).all()
    return o


@pytest.mark.parametrize("R,d", [(512, 128), (256, 64), (512, 64), (256, 128)])
@pytest.mark.parametrize("H,block", [(1, 16), (3, 64), (2, 5), (2, 640)])
def test_latent_prefill(R, d, H, block):
    say(f"case latent prefill R={R} d={d} H={H} block={block}")
    _check_prefill(_prefill_case(R + d + H, [0, 0, 70, 5, 0, 130], [1, 130, 3, 0, 65, 40], H, R,
                                 d, block))


@pytest.mark.parametrize("n", [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 257])
def test_latent_prefill_lengths(n):
    say(f"case latent prefill length {n}")
    _check_prefill(_prefill_case(n, [0], [n], 2, 256, 64, 64))


@pytest.mark.parametrize("ctx,new", [([900], [1]), ([700], [100]), ([0], [900]), ([1], [300])])
def test_latent_prefill_long_rows(ctx, new):
    say(f"case latent prefill long {ctx} {new}")
    _check_prefill(_prefill_case(9, ctx, new, 2, 512, 128, 64), every=5)


def test_latent_prefill_many_sequences():
    say("case latent prefill n=300")
    g = gen(5)
    new = torch.randint(0, 7, (300,), generator=g).tolist()
    ctx = torch.randint(0, 30, (300,), generator=g).tolist()
    _check_prefill(_prefill_case(6, ctx, new, 1, 256, 64, 16), every=3)


@pytest.mark.parametrize("block", [8, 64, 100])
def test_latent_prefill_null_blocks(block):
    """Null entries, ids past the pool; a request whose first rows see nothing."""
    say(f"case latent prefill null {block}")
    case = list(_prefill_case(9, [60, 0, 0], [200, 130, 20], 2, 512, 128, block))
    case[4][0, 0] = -1
    case[4][0, 1] = 1 << 30
    case[4][1, 0] = -9
    case[4][2, :] = -1
    o = _check_prefill(tuple(case), every=3)
    assert torch.equal(o[330:], torch.zeros_like(o[330:]))
    assert torch.equal(o[200], torch.zeros_like(o[200]))


def test_latent_prefill_more_new_tokens_than_the_length():
    """seq_lens below the packed rows: the first rows lie before the request's start."""
    say("case latent prefill new > len")
    case = list(_prefill_case(10, [0, 0], [40, 10], 2, 256, 64, 16, poison=False))
    case[6] = torch.tensor([25, 0], dtype=torch.int32)
    o = _check_prefill(tuple(case))
    assert torch.equal(o[:15], torch.zeros_like(o[:15]))
    assert torch.equal(o[40:], torch.zeros_like(o[40:]))


def test_latent_prefill_leaves_rows_behind_the_last_sequence():
    say("case latent prefill padded")
    case = list(_prefill_case(11, [0, 20], [70, 33], 2, 256, 64, 16))
    want = _run_prefill(tuple(case))
    pad = [torch.cat([x, torch.full((50, *x.shape[1:]), float("nan"), dtype=BF16)])
           for x in case[:2]]
    o = torch.full((153, 2, 64), 7.0, dtype=BF16, device=DEV)
    got = _run_prefill((*pad, *case[2:]), keys=1000, o=o)
    assert torch.equal(got[:103], want)
    assert torch.equal(got[103:], torch.full_like(got[103:], 7.0))


def test_latent_prefill_with_too_few_keys_stays_inside():
    """A total_keys below the lengths loses keys: outputs of the requests before are right."""
    say("case latent prefill short total_keys")
    case = _prefill_case(12, [0, 0], [100, 300], 2, 256, 64, 16, poison=False)
    full = _run_prefill(case)
    got = _run_prefill(case, keys=128)
    assert torch.equal(got[:100], full[:100]) and torch.isfinite(got.float()).all()


def test_latent_prefill_equals_decode_token_by_token():
    """The two forms of the same attention agree to rounding."""
    say("case latent prefill vs decode")
    case = _prefill_case(13, [37], [9], 4, 512, 128, 16, poison=False)
    a = _run_prefill(case).float()
    qn, qp, w, cache, table, cu, lens, scale = case
    b = gdn.gdn_latent_decode(qn[None].to(DEV), qp[None].to(DEV), w.to(DEV), cache.to(DEV),
                              table.to(DEV), lens.to(DEV), scale=scale)[0].float()
    torch.cuda.synchronize()
    # each is within its roundings (a few half steps of 2^-8) of the same value
    assert (a - b).abs().max() <= 0.05 * b.abs().max()
