"""The decode kernels where a worker takes many key chunks of a unit in a row, under scores that
outgrow the running reference again and again: what a new reference scales older sums and outputs
by. Each case works out from the split's own rule how many chunks a worker takes, so that it
cannot come down to one chunk a worker, whose sums are never rescaled."""
import numpy as np
import pytest
import torch

import test_gpu_latent as lat
import test_gpu_paged as pag
from attn_util import assert_within, tolerance
from gpu_util import say
from oracle import attention

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ROPE = 64
BLOCK = 64


def _cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _workers(workgroups, row_tiles):
    return min(max(workgroups // row_tiles // 8 * 8, 8), 1024)


def _paged_run(lens, P, H, kv, d, dtype):
    """(16-row tiles a workgroup holds, chunks of a worker) of gdn_paged_decode."""
    tiles = -(-P * (H // kv) // 16)
    most = 1 if dtype is F32 or d == 256 else 2 if d == 128 else 4
    rt = 4 if tiles >= 4 and most >= 4 else 2 if tiles >= 2 and most >= 2 else 1
    row_tiles = -(-tiles // rt)
    keys = 4 * (32 if dtype is BF16 and d < 256 else 16)
    total = sum(-(-n // keys) + 2 for n in lens) * kv
    two = rt == 1 and (dtype is BF16 or d <= 128)
    workers = _workers((2 if two else 1) * _cus(), row_tiles)
    if two and row_tiles == 1 and total // 8 >= len(lens) * kv:
        workers //= 2
    return rt, total // workers


def _latent_run(lens, P, H):
    """The same for gdn_latent_decode."""
    tiles = -(-P * H // 16)
    rt = 4 if tiles > 2 else tiles
    workers = _workers(_cus(), -(-tiles // rt))
    return rt, sum(-(-n // 64) + 6 for n in lens) // workers


def _ramp(n, kind):
    """Whole numbers below 2^16. Under the scales below neighbours differ by less than the lag of
    the reference, runs of some dozens of keys by more."""
    j = torch.arange(n)
    if kind == "rising":
        return j
    if kind == "falling":
        return n - 1 - j
    if kind == "steps":                       # flat for 200 keys, then far above them
        return j // 200 * 150
    return j % 517 // 3 + (j % 1300 == 700) * 400 + j // 900 * 90   # waves, spikes, a slow rise


def _parts(x):
    """x as a sum of two numbers that bf16 holds exactly (|x| < 2^16, whole)."""
    low = torch.remainder(x, 256)
    return low.to(BF16), (x - low).to(BF16)


KINDS = ["rising", "falling", "steps", "waves"]
FACTORS = torch.tensor([1.0, -1.0, 0.5, 2.0, -0.25])   # of the rows: exact in bf16


def _row_factors(*shape):
    """Neighbouring rows differ, and so do the rows of one column over the tiles."""
    n = int(np.prod(shape))
    i = torch.arange(n)
    return FACTORS[(i + i // 5) % 5].view(shape)


def _put(write, table, lens, at):
    """A ramp of another kind for every request, in two columns of its tokens' rows:
    write(page, offset, column, values)."""
    for i, n in enumerate(lens):
        j = torch.arange(n)
        low, high = _parts(_ramp(n, KINDS[i % 4]))
        page, off = table[i][j // BLOCK].long(), j % BLOCK
        write(page, off, at[0], low)
        write(page, off, at[1], high)


# ------------------------------------------------------------------------------ grouped heads
@pytest.mark.parametrize("dtype,d,H,kv,P,lens", [
    (BF16, 64, 8, 8, 1, [8000, 7930, 6400, 8001, 5000]),     # one row tile, many units
    (BF16, 128, 16, 8, 1, [8000, 7930, 6400, 8001, 5000]),
    (BF16, 256, 8, 4, 2, [8000, 7930, 6400, 8001, 5000]),
    (BF16, 128, 160, 1, 4, [4000, 5100, 2900, 3003]),        # tiles of 32 rows, 20 of them
    (BF16, 64, 160, 1, 8, [4000, 5100, 2900, 3003]),         # tiles of 64 rows, 20 of them
    (BF16, 256, 160, 1, 2, [3000, 3100, 2500, 2002]),        # 16 rows, 20 tiles
    (F32, 64, 8, 8, 1, [4000, 3930, 3200, 4001, 2500]),
    (F32, 128, 160, 1, 2, [3000, 3100, 2500, 2002]),
    (F32, 256, 40, 2, 4, [3000, 3100, 2500, 2002])])
def test_paged_decode_rescales_over_many_chunks(dtype, d, H, kv, P, lens):
    rt, chunks = _paged_run(lens, P, H, kv, d, dtype)
    say(f"case long runs paged {dtype} d={d} H={H} kv={kv} P={P}: tiles of {16 * rt} rows, "
        f"{chunks} chunks a worker")
    assert chunks >= 4
    case = list(pag._decode_case(d + H, lens, P, H, kv, d, BLOCK, dtype, poison=False))
    q, kc, vc, table = case[:4]
    kc.zero_()

    def write(page, off, col, x):
        kc[page, :, off, col] = x[:, None].to(dtype)
    _put(write, table, lens, (3, d - 7))
    q.zero_()
    q[..., 3] = q[..., d - 7] = _row_factors(len(lens), P, H).to(dtype)
    heads = list(range(0, H, max(H // 16, 1)))             # the reference's share of them
    used = sorted({h // (H // kv) for h in heads})
    assert [h // (H // kv) for h in heads] == [used[i * len(used) // len(heads)]
                                               for i in range(len(heads))]
    for scale in (0.11, -0.11):
        case[5] = scale
        o = pag._run_decode(tuple(case))
        want, mag, top = attention.paged_decode(q[:, :, heads], kc[:, used], vc[:, used], table,
                                                case[4], scale)
        assert_within(o[:, :, heads], want, tolerance(want, mag, top, d, max(lens), dtype),
                      f"scale {scale}")


# -------------------------------------------------------------------------------------- latent
@pytest.mark.parametrize("H,P,R,lens", [
    (4, 1, 256, [20000, 19990, 18000, 16001]),               # tiles of 16 rows
    (8, 1, 512, [20000, 19990, 18000, 16001]),
    (10, 2, 256, [20000, 19990, 18000, 16001]),              # of 32
    (64, 8, 256, [4000, 5100, 2900, 3003]),                  # of 64, 8 of them
    (64, 8, 512, [4000, 5100, 2900, 3003])])
def test_latent_decode_rescales_over_many_chunks(H, P, R, lens):
    rt, chunks = _latent_run(lens, P, H)
    say(f"case long runs latent H={H} P={P} R={R}: tiles of {16 * rt} rows, {chunks} chunks a "
        "worker")
    assert chunks >= 4
    case = list(lat._decode_case(H + R, lens, P, H, R, 64, BLOCK, poison=False))
    qn, qp, w, cache, table, ln, _ = case
    cache[..., R:] = 0.0

    def write(page, off, col, x):
        cache[page, off, R + col] = x
    _put(write, table, lens, (0, 5))
    qn.zero_()
    qp.zero_()
    qp[..., 0] = qp[..., 5] = _row_factors(len(lens), P, H).to(BF16)
    # the reference's share of the rows
    heads, at = sorted({0, 1, H // 2, H - 1}), sorted({0, P - 1})
    for scale in (0.11, -0.11):
        case[6] = scale
        o = lat._run_decode(tuple(case))
        for b in range(len(lens)):
            part = [qn[b:b + 1][:, :, heads], qp[b:b + 1][:, :, heads], w[heads], cache,
                    table[b:b + 1]]
            want = attention.latent_absorbed(*part, ln[b:b + 1], scale)[0, at]
            tol = lat._tolerance(part[0][0, at], part[1][0, at], *part[2:],
                                 [(0, lens[b] - P + p + 1) for p in at], want, scale)
            assert_within(o[b][at][:, heads], want, tol, f"request {b}, scale {scale}")
