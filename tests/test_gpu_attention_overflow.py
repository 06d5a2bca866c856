"""A step whose new tokens exceed its buffers: gdn_paged_plan leaves the tokens behind max_tokens
without a slot and says so in counts[0]; its cu_seqlens count them all the same. The rows that
have their place keep their positions in gdn_latent_prefill."""
import numpy as np
import pytest
import torch

import test_gpu_latent as lat
from attn_util import assert_within, gen, normal, pages
from gated_delta_rule_prefill_amd import gdn
from gpu_util import DEV, say
from oracle import attention

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32
ROPE, R, D, H, BLOCK = 64, 256, 64, 2, 16
SCALE = (D + ROPE) ** -0.5


def ints(x):
    return torch.tensor(x, dtype=I32, device=DEV)


def _step(seed, ctx, new, rows):
    """Plan and append of a step into buffers of `rows` tokens; slots that no token was written to
    hold NaN. Returns everything a prefill call takes, on the GPU."""
    g = gen(seed)
    lens = [c + w for c, w in zip(ctx, new)]
    table, n_blocks = pages(g, lens, BLOCK)
    held = torch.tensor([-(-c // BLOCK) for c in ctx])
    fresh = torch.arange(table.shape[1])[None] >= held[:, None]
    free = table[fresh]
    free = free[free >= 0].to(DEV)
    cache = torch.full((n_blocks, BLOCK, R + ROPE), float("nan"), dtype=BF16)
    for i, c in enumerate(ctx):
        j = torch.arange(c)
        cache[table[i][j // BLOCK].long(), j % BLOCK] = normal(g, c, R + ROPE)
    table[fresh] = -1
    table, cache = table.to(DEV), cache.to(DEV)
    cu, ln, slots, pos, counts = gdn.gdn_paged_plan(ints(ctx), ints(new), table, free, BLOCK, rows)
    gdn.gdn_latent_append(normal(g, rows, R).to(DEV), normal(g, rows, ROPE).to(DEV), slots, cache)
    assert int(counts[0]) == sum(new)
    qn, qp = normal(g, rows, H, D, scale=1.5).to(DEV), normal(g, rows, H, ROPE, scale=1.5).to(DEV)
    return qn, qp, lat._weights(g, H, R, D).to(DEV), cache, table, cu, ln, pos


@pytest.mark.parametrize("ctx,new,rows", [
    ([20, 5, 9], [30, 40, 7], 50), ([20, 5, 9], [30, 40, 7], 31), ([20, 5, 9], [30, 40, 7], 30),
    ([20, 5, 9], [30, 40, 7], 1), ([0, 70], [200, 300], 350), ([0], [300], 129), ([3], [2], 1)])
def test_rows_before_the_cut_keep_their_positions(ctx, new, rows):
    say(f"case prefill of a cut step {ctx} {new} {rows}")
    qn, qp, w, cache, table, cu, ln, pos = _step(1, ctx, new, rows)
    o = gdn.gdn_latent_prefill(qn, qp, w, cache, table, cu, ln, sum(ctx) + sum(new), scale=SCALE)
    # the same step without the tokens that were cut off
    kept = [min(w_, max(rows - at, 0)) for w_, at in zip(new, np.cumsum([0] + new[:-1]).tolist())]
    short = [c + k for c, k in zip(ctx, kept)]
    cu_short = [0] + np.cumsum(kept).tolist()
    assert pos.tolist() == [p for c, k in zip(ctx, kept) for p in range(c, c + k)]
    same = gdn.gdn_latent_prefill(qn, qp, w, cache, table, ints(cu_short), ints(short), sum(short),
                                  scale=SCALE)
    torch.cuda.synchronize()
    host = [x.cpu() for x in (qn, qp, w, cache, table)]
    clean = torch.nan_to_num(host[3].float()).double()
    want = attention.latent_expanded(*host[:3], clean, host[4], cu_short, short, SCALE)
    limits = [(i, c + t + 1) for i, (c, k) in enumerate(zip(ctx, kept)) for t in range(k)]
    pick = list(range(0, rows, 3))
    tol = lat._tolerance(host[0][pick], host[1][pick], host[2], host[3], host[4],
                         [limits[t] for t in pick], want[pick], SCALE)
    assert_within(o[pick], want[pick], tol)
    assert torch.equal(o, same)
