"""The main loop of paged_attend.h once its buffers have gone round several times: runs of 20 steps
and more for every worker, with odd page sizes, null pages among them, and requests of other
lengths. Queries are long, so that a row's softmax rests on a few of its keys, and the rows' few
keys lie in all steps: a step that is left out, taken twice or read from other pages shows in the
rows that rest on it."""
import pytest
import torch

import test_gpu_paged_prefill as pre
import test_gpu_shared_decode as sha
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
TYPES = [(BF16, 64), (BF16, 128), (BF16, 256), (F32, 64)]


def steps_a_worker(units, dtype):
    """units: keys that each (tile, key/value head) reaches."""
    step = 64 if dtype == BF16 else 32
    workers = torch.cuda.get_device_properties(0).multi_processor_count // 8 * 8
    return sum(-(-n // step) for n in units) / workers


def drop_pages(table, rows, every):
    """Null pages in the middle of runs, one and two at a time."""
    for i in rows:
        table[i, every::every] = -1
        table[i, every + 1::3 * every] = -1


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("block,null", [(48, False), (20, True)])
def test_prompts(gpu_lib, block, null, dtype, d):
    lens, new, H, kv = [16000, 15555, 14001, 70], [60, 90, 33, 70], 8, 8
    say("long runs", dtype, d, block, null)
    assert steps_a_worker([n for n in lens for _ in range(kv)], dtype) >= 20
    args = list(pre.make(80, lens, new, H, kv, d, block, dtype))
    args[0] *= 4
    if null:
        drop_pages(args[3], (0, 2), 17)
    pre.check(gpu_lib, args, d ** -0.5, "long runs")


def test_prompts_of_several_tiles(gpu_lib):
    """Causal tiles: waves whose rows end before the workgroup's last step."""
    lens, new, H, kv = [5200, 3000], [1100, 900], 8, 4
    assert steps_a_worker([n - w + min(t + 128, w) for n, w in zip(lens, new)
                           for t in range(0, w, 128) for _ in range(kv)], BF16) >= 15
    args = list(pre.make(81, lens, new, H, kv, 64, 24, BF16))
    args[0] *= 4
    pre.check(gpu_lib, args, 0.125, "several tiles")


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("block,null", [(64, True), (24, False)])
def test_shared_prefixes(gpu_lib, block, null, dtype, d):
    prefix, kv = [16000, 14500, 9001], 8
    say("long shared runs", dtype, d, block, null)
    assert steps_a_worker([n for n in prefix for _ in range(kv)], dtype) >= 18
    args = list(sha.make(82, [2, 3, 2], prefix, [5, 40, 9, 1, 300, 20, 77], 1, 8, kv, d, block, dtype,
                         part=False))
    args[0] *= 4
    if null:  # (the rows of a group name the same pages)
        drop_pages(args[3], (0, 1), 19)
    sha.check(gpu_lib, args, d ** -0.5, "long shared runs")


def test_a_shared_prefix_of_several_tiles(gpu_lib):
    """20 requests of 16 positions: a head's two tiles read the same keys at the same time."""
    args = list(sha.make(83, [20], [6000], [16 + i % 7 for i in range(20)], 16, 16, 16, 64, 32, BF16,
                         part=False))
    assert steps_a_worker([6000] * 32, BF16) >= 11
    args[0] *= 4
    sha.check(gpu_lib, args, 0.125, "two tiles")
