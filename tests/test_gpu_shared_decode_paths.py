"""Which form gdn_paged_shared_decode takes, made visible: the rows of a group's later requests name
other pages than its first for the prefix, which the contract does not allow, so that a result
tells whose pages were read. Prefixes attended apart come from the first row (for all requests
of the group); requests that read their own give plain decode over their own rows."""
import pytest
import torch

from attn_util import assert_within, gen, normal, tolerance
from gpu_util import DEV, say
from oracle import attention, pages as oracle_pages

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
MIB = 1 << 20


def make(seed, sizes, prefix, H, kv, d, block, dtype, own=7, loose=1):
    """Groups whose rows name pages of their own throughout; all prefixes are whole pages."""
    g = gen(seed)
    B = sum(sizes) + loose
    cu, skip = [0], []
    for s, x in zip(sizes, prefix):
        cu.append(cu[-1] + s)
        skip += [x] * s
    lens = [x + own for x in skip + [0] * loose]
    width = -(-max(lens) // block)
    # each row names a few pages of its own many times over
    n = 12
    table = torch.randint(n, (B, width), generator=g, dtype=torch.int32)
    table += n * torch.arange(B, dtype=torch.int32)[:, None]
    k, v = (normal(g, n * B, kv, block, d, dtype=dtype) for _ in range(2))
    q = normal(g, B, 1, H, d, dtype=dtype, scale=4.0)
    return (q, k, v, table, torch.tensor(lens, dtype=torch.int32),
            torch.tensor(cu, dtype=torch.int32), torch.tensor(prefix, dtype=torch.int32))


def spared(sizes, prefix, kv, d, dtype):
    return sum((s - 1) * x for s, x in zip(sizes, prefix)) * 2 * kv * d * dtype.itemsize


class Case:
    def __init__(self, lib, args, scale):
        self.lib, self.scale = lib, scale
        q, k, v, table, lens, cu, prefix = args
        self.dev = [x.to(DEV) for x in args]
        n = max(int(lens.max()), 1)

        def with_tolerance(want, mag, top):
            return want, tolerance(want, mag, top, q.shape[3], n, q.dtype)
        kf, vf = k.float(), v.float()
        self.apart = with_tolerance(*oracle_pages.shared_decode(q, kf, vf, table, lens, cu, prefix,
                                                                scale))
        self.own = with_tolerance(*attention.paged_decode(q, kf, vf, table, lens, scale))
        # the two differ by more than both tolerances, or the case shows nothing
        far = abs(self.apart[0] - self.own[0]) > self.apart[1] + self.own[1]
        assert far.mean() > 0.2, far.mean()

    def takes(self, form, **kw):
        o = self.lib.gdn_paged_shared_decode(*self.dev, scale=self.scale, **kw)
        want, tol = self.apart if form == "apart" else self.own
        assert_within(o, want, tol, f"{form} {kw}")
        return o


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 128), (BF16, 256), (F32, 64), (F32, 128),
                                     (F32, 256)])
def test_the_least_that_the_caller_names(gpu_lib, dtype, d):
    sizes, prefix, H, kv, block = [3, 1, 4], [96, 64, 160], 8, 2, 16
    say("paths", dtype, d)
    case = Case(gpu_lib, make(1, sizes, prefix, H, kv, d, block, dtype), d ** -0.5)
    n = spared(sizes, prefix, kv, d, dtype)
    for least in (0, 1, n - 1, n):
        case.takes("apart", min_bytes=least)
    for least in (n + 1, 2 ** 62):
        case.takes("own", min_bytes=least)
    case.takes("own")                       # far below what the library's rule asks for


# (dtype, d, group sizes, KV heads, heads, page size, least): prefixes as long as it takes to come to
# the least, and one page shorter
RULE = [(BF16, 128, [33], 4, 8, 16, 128 * MIB), (BF16, 256, [9, 9], 2, 4, 32, 128 * MIB),
        (F32, 64, [65], 2, 2, 64, 256 * MIB)]


@pytest.mark.parametrize("case", range(len(RULE)))
def test_the_library_rule_at_its_threshold(gpu_lib, case):
    dtype, d, sizes, kv, H, block, least = RULE[case]
    per_block = spared(sizes, [block] * len(sizes), kv, d, dtype)
    blocks = -(-least // per_block)
    for n, form in ((blocks, "apart"), (blocks - 1, "own")):
        prefix = [n * block] * len(sizes)
        assert (spared(sizes, prefix, kv, d, dtype) >= least) == (form == "apart")
        say("rule", dtype, d, sizes, prefix, form)
        c = Case(gpu_lib, make(2 + case, sizes, prefix, H, kv, d, block, dtype), d ** -0.5)
        assert torch.equal(c.takes(form), c.takes(form, min_bytes=0 if form == "apart" else 2 ** 62))


@pytest.mark.parametrize("sizes,H,kv,form", [([2], 128, 4, "apart"), ([3], 63, 3, "own")])
def test_fp32_groups_need_64_rows(gpu_lib, sizes, H, kv, form):
    """64 and 63 rows of a key/value head, 270 MiB spared."""
    d, block = 256, 16
    n = -(-270 * MIB // spared(sizes, [block], kv, d, F32))
    c = Case(gpu_lib, make(7, sizes, [n * block], H, kv, d, block, F32, loose=0), d ** -0.5)
    c.takes(form)
    c.takes("apart", min_bytes=0)


def test_groups_of_one_and_prefixes_of_none_read_their_own(gpu_lib):
    args = list(make(8, [1, 2, 1], [64, 48, 32], 4, 2, 64, 16, BF16))
    args[6][1] = 0                          # the only group of two names no tokens
    q, k, v, table, lens = args[:5]
    want, mag, top = attention.paged_decode(q, k.float(), v.float(), table, lens, 0.125)
    o = gpu_lib.gdn_paged_shared_decode(*(x.to(DEV) for x in args), scale=0.125, min_bytes=0)
    assert_within(o, want, tolerance(want, mag, top, 64, 80, BF16), "nothing shared")
