"""gdn_paged_copy where a pair names one page twice: such a pair is none, as the debug library has
it, and leaves the page to the pair that writes it."""
import pytest
import torch

from gated_delta_rule_prefill_amd import gdn
from gpu_util import DEV
from test_gpu_debug_checks import debug_lib
from test_gpu_shared_run import ints

pytestmark = pytest.mark.gpu


def pools(n_blocks, page):
    """A pool of small pages and one of pages that take several workgroups each."""
    return [torch.arange(n_blocks * page * k, dtype=torch.int32, device=DEV).view(n_blocks, page * k)
            for k in (1, 3)]


@pytest.mark.parametrize("page", [4, 5000])
@pytest.mark.parametrize("order", [1, -1])
def test_a_page_and_itself_is_no_pair(gpu_lib, page, order):
    src, dst = [5, 3, 7, 6, 1, 9], [5, 5, 7, 8, 1, 1]
    for c in pools(10, page):
        want = c.clone()
        for a, b in zip(src, dst):
            want[b] = c[a] if a != b else want[b]
        gpu_lib.gdn_paged_copy([c], ints(src[::order]), ints(dst[::order]))
        assert torch.equal(c, want)


def test_the_debug_library_takes_them_as_none(gpu_lib):
    c = torch.arange(40, dtype=torch.float32, device=DEV).view(10, 4)
    want = c.clone()
    want[5], want[6] = c[3], c[7]
    with debug_lib():
        gdn.gdn_paged_copy([c], ints([5, 3, 7, 7]), ints([5, 5, 7, 6]))
        assert torch.equal(c, want)
        with pytest.raises(gdn.GdnError, match="source"):
            gdn.gdn_paged_copy([c], ints([5, 3, 5]), ints([5, 5, 2]))
    assert torch.equal(c, want)


def test_a_fork_of_no_rows_passes_the_debug_library(gpu_lib):
    none, one = ints([]), ints([[1, 2]])
    with debug_lib():
        a, b, counts = gdn.gdn_paged_fork(none, none, none, one, 16, ints([0] * 4), ints([3]))
    assert a.numel() == b.numel() == 0 and counts.cpu().tolist() == [0, 0]
