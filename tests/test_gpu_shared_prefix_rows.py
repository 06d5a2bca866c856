"""gdn_paged_shared_decode where the requests of a group end, the first of them too: the prefix
is read from a row that still holds it. Against the fp64 oracle of plain decode attention, in which
every request reads its own row."""
import pytest
import torch

import test_gpu_shared_decode as sha
from attn_util import assert_within, gen, normal, tolerance
from gpu_util import DEV, say
from oracle import attention
from test_gpu_shared_run import Engine, ints

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def end(args, rows, block):
    """Requests that ended and stay in the batch as padded rows: no tokens, no pages."""
    for b in rows:
        args[3][b], args[4][b] = -1, 0


def cut(args, rows, lens, block):
    """Requests of fewer tokens, whose later entries name no page."""
    for b, n in zip(rows, lens):
        args[3][b, -(-n // block):], args[4][b] = -1, n


def check(lib, args, scale, what):
    q, k, v, table, lens, cu, prefix = args
    dev = [x.to(DEV) for x in args]
    want, mag, top = attention.paged_decode(q, torch.nan_to_num(k.float()),
                                            torch.nan_to_num(v.float()), table, lens, scale)
    tol = tolerance(want, mag, top, q.shape[3], max(int(lens.max()), 1), q.dtype)
    for least in (0, 2 ** 62, -1):
        o = lib.gdn_paged_shared_decode(*dev, scale=scale, min_bytes=least)
        assert_within(o, want, tol, f"{what}, least {least}")
    return o


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 128), (BF16, 256), (F32, 64)])
@pytest.mark.parametrize("gone", [[0], [0, 1, 2], [1, 4], [0, 1, 2, 3, 4]])
def test_ended_requests_of_a_group(gpu_lib, gone, dtype, d):
    say("ended", gone, dtype, d)
    args = list(sha.make(40, [5, 3], [300, 90], [7, 9, 30, 2, 70, 1, 2, 3], 1, 8, 2, d, 16, dtype))
    end(args, gone, 16)
    o = check(gpu_lib, args, d ** -0.5, "ended")
    assert bool((o[gone] == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens", [[40, 307, 200], [40, 16, 200], [0, 0, 17], [299, 300, 301],
                                  [0, 3, 3]])
def test_requests_that_hold_a_part_of_the_prefix(gpu_lib, lens, dtype):
    """The longest request of a group that nobody holds all of; verify steps of 3 positions."""
    args = list(sha.make(41, [3, 2], [300, 50], [9] * 5, 3, 4, 2, 64, 16, dtype))
    cut(args, range(3), lens, 16)
    check(gpu_lib, args, 0.125, f"lengths {lens}")


@pytest.mark.parametrize("dtype,gone", [(BF16, range(64)), (BF16, range(60)), (F32, range(33))])
def test_tiles_whose_requests_all_ended(gpu_lib, dtype, gone):
    """70 requests of 4 rows: tiles of 64 and 32 of them."""
    args = list(sha.make(42, [70], [130], [3] * 70, 1, 8, 2, 64, 16, dtype))
    end(args, gone, 16)
    check(gpu_lib, args, 0.125, "tiles")


@pytest.mark.parametrize("dtype,d,block", [(BF16, 128, 16), (F32, 64, 24)])
def test_a_run_in_which_the_parent_ends(gpu_lib, dtype, d, block):
    """A prompt, four samples of it, steps; the prompt's own request ends and stays in the batch;
    further steps behind the prefix, which the samples still hold."""
    H, kv, rows = 8, 2, 5
    e = Engine(rows, 30, 120, block, H, kv, d, dtype, 71)
    e.step([150, 0, 0, 0, 0], e.prefill)
    a, b, counts = gpu_lib.gdn_paged_fork(ints([0] * 4), ints([1, 2, 3, 4]), ints([150] * 4), e.table,
                                          block, e.shares, e.free)
    gpu_lib.gdn_paged_copy([e.kc, e.vc], a, b)
    e.take(int(counts[1]))
    for t in range(1, rows):
        e.lens[t], e.held[t] = 150, e.held[0]
    cu, prefix = ints([0, rows]), ints([150 // block * block])

    def shared(q, _, lens):
        T = q.shape[0] // len(running)
        padded = torch.zeros(rows, T, H, d, dtype=dtype, device=DEV)
        padded[running] = q.view(len(running), T, H, d)
        o = gpu_lib.gdn_paged_shared_decode(padded, e.kc, e.vc, e.table, lens, cu, prefix,
                                            scale=e.scale, min_bytes=0)
        return o[running]
    running = list(range(rows))
    e.step([1] * rows, shared)
    gpu_lib.gdn_paged_free(ints([0]), ints([e.lens[0]]), e.table, block, e.shares)
    assert bool((e.table[0] == -1).all())
    e.lens[0], e.held[0] = 0, e.held[0][:0]
    running = [1, 2, 3, 4]
    for P in (1, 2):
        e.step([0] + [P] * 4, shared)
