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
