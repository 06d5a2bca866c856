"""gdn_latent_prefill where a workgroup of its expanding launch forms several runs of 512 columns
of keys and values one after the other: each run's first weights are requested while the run
before it ends, and the last run may be a partial one."""
import pytest
import torch

import test_gpu_latent as lat
from gpu_util import say

pytestmark = pytest.mark.gpu


def runs_of_a_workgroup(ctx, new, H, d):
    """The launch's choice for total_keys = the sum of the lengths: (columns in 512s, runs of a
    workgroup)."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    keys = sum(ctx) + sum(new)
    blocks = ((keys + 63 * len(ctx)) // 64 + 1) // 2
    units = -(-H * 2 * d // 512)
    cost = {}
    for workgroups in range(1, units + 1):
        n = -(-units // workgroups)
        cost.setdefault(-(-blocks * workgroups // cus) * (3 * n + 1), n)
    return units, cost[min(cost)]


@pytest.mark.parametrize("R,H,d,ctx,new", [
    (512, 32, 128, [3300, 790, 0], [5, 3, 2]),      # 16 runs of columns, 3 a workgroup: 5 x 3 + 1
    (256, 33, 128, [4100, 0, 20], [4, 1, 3]),       # an odd head at the end: half a run
    (512, 21, 64, [6000, 300], [4, 3]),             # runs of four heads, a quarter of one left
    (256, 21, 64, [2500, 3700], [2, 4]),
    (512, 5, 128, [23000, 100], [3, 4]),            # every run in one workgroup
])
def test_columns_in_several_runs(R, H, d, ctx, new):
    say(f"case latent prefill runs R={R} H={H} d={d} {ctx}")
    units, per = runs_of_a_workgroup(ctx, new, H, d)
    assert per > 1, (units, per)
    lat._check_prefill(lat._prefill_case(R + H, ctx, new, H, R, d, 64), every=2)
