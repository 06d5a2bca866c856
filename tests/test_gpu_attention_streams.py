"""Buffers that the binding of the attention calls makes for a stream given by its handle."""
import pytest
import torch

import test_gpu_paged as pag
from gated_delta_rule_prefill_amd import gdn
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def _stream_of(t):
    """Handle of the stream whose memory holds a tensor."""
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the caching allocator's")


@pytest.mark.parametrize("which", ["default", "default handle", "side", "side handle"])
def test_results_come_from_the_given_streams_memory(which):
    """Handle 0 is the default stream, whose queued work may still use what is freed here."""
    say(f"case stream memory {which}")
    q, kc, vc, table, lens, scale = (x.to(DEV) if torch.is_tensor(x) else x for x in
                                     pag._decode_case(1, [40, 7], 1, 4, 2, 64, 16, torch.bfloat16))
    want = gdn.gdn_paged_decode(q, kc, vc, table, lens, scale=scale)
    torch.cuda.synchronize()
    stream = torch.cuda.default_stream() if "default" in which else torch.cuda.Stream()
    given = stream.cuda_stream if "handle" in which else stream
    assert "default" not in which or stream.cuda_stream == 0
    with torch.cuda.stream(torch.cuda.Stream()):
        o = gdn.gdn_paged_decode(q, kc, vc, table, lens, scale=scale, stream=given)
    torch.cuda.synchronize()
    assert torch.equal(o, want)
    assert _stream_of(o) == stream.cuda_stream
