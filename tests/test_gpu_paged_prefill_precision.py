"""What gdn_paged_prefill and the prefixes of gdn_paged_shared_decode lose between bf16 inputs and
the rounding of their outputs, over all outputs together: the 2-norm of the error against the fp64
reference, in terms of e0, that of the reference rounded to bf16 once.

Derivation. With weights p_i of the sum L and relative roundings d_i, independent and as large as
e0 (a bf16 number's relative error is spread over the half step alike for outputs and weights),
  sum (1 + d_i) p_i v_i / sum (1 + d_i) p_i = o + sum d_i p_i (v_i - o) / L + higher orders,
so the weights' roundings add e0^2 sum (p_i / L)^2 |v_i - o|^2 to the square of the error. For two
keys that is 2 e0^2 (p / (1 + p)^2)^2 |v_1 - v_0|^2, p their ratio; for many keys and zero-mean
values at most the expected e0^2 |o|^2. 5 % on top for the spread over the inputs drawn."""
import numpy as np
import pytest
import torch

import test_gpu_paged_prefill as pre
import test_gpu_shared_decode as sha
from attn_util import gen, normal
from gpu_util import DEV, say
from oracle import pages as oracle_pages

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def errors(got, want):
    """(2-norm of the error, the same of the reference rounded to bf16 once)."""
    once = torch.from_numpy(want).to(BF16).double().numpy()
    return np.linalg.norm(got.double().cpu().numpy() - want), np.linalg.norm(once - want)


def two_keys(seed, requests, new, d):
    """Requests of 64 + 4 + new tokens, of whose keys two count: one in the first 64 and one
    behind them, 0.4 to 7.6 powers of two above it, which is within what the reference of the
    exponents lags behind. All others lie 200 below. (More requests than workers, so that most
    requests are attended by one worker.)"""
    g = gen(seed)
    n, block = 68 + new, 16
    pages = -(-n // block)
    k = torch.zeros(requests * pages, 1, block, d, dtype=BF16)
    v = normal(g, requests * pages, 1, block, d)
    k[:, 0, :, 2] = -200
    table = torch.arange(requests * pages, dtype=torch.int32).view(requests, pages)
    first, second = table[:, 1].long(), table[:, 4].long()    # tokens 21 and 65
    k[first, 0, 5], k[second, 0, 1] = 0, 0
    k[first, 0, 5, 0], k[second, 0, 1, 1] = 1, 1
    q = torch.zeros(requests * new, 1, d, dtype=BF16)
    q[:, 0, 0], q[:, 0, 2] = 1, 1
    q[:, 0, 1] = (1 + 0.3 + 5 * torch.rand(requests * new, generator=g)).to(BF16)
    cu = torch.arange(requests + 1, dtype=torch.int32) * new
    return q, k, v, table, cu, torch.full((requests,), n, dtype=torch.int32)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_weight_that_outweighs_the_others_is_exact(gpu_lib, d):
    requests, new = 700, 2
    args = two_keys(d, requests, new, d)
    q, k, v, table, cu, lens = args
    o = gpu_lib.gdn_paged_prefill(*(x.to(DEV) for x in args), scale=1.0)
    want, _, _ = oracle_pages.prefill(q, k.float(), v.float(), table, cu, lens, 1.0)
    e, e0 = errors(o, want)
    p = np.exp(q[:, 0, 1].double().numpy() - 1)
    v0, v1 = (v[table[:, c].long(), 0, r].double().numpy().repeat(new, axis=0)
              for c, r in ((1, 5), (4, 1)))
    assert np.abs(want[:, 0] - (v0 + p[:, None] * v1) / (1 + p[:, None])).max() < 1e-12
    unit = e0 / np.linalg.norm(want)
    lost = unit ** 2 * 2 * ((p / (1 + p) ** 2) ** 2 * ((v1 - v0) ** 2).sum(axis=1)).sum()
    say(f"case two keys d={d}: {e / e0:.4f}, at most {1.05 * np.sqrt(1 + lost / e0 ** 2):.4f}")
    assert e <= 1.05 * np.sqrt(e0 ** 2 + lost)


@pytest.mark.parametrize("d,H,kv,lens,new", [
    (128, 8, 2, [700, 600], [700, 600]), (64, 8, 4, [1500, 900], [300, 200]),
    (256, 4, 2, [900, 300], [200, 300])])
def test_prompts_lose_little(gpu_lib, d, H, kv, lens, new):
    args = pre.make(d + 1, lens, new, H, kv, d, 32, BF16)
    o = gpu_lib.gdn_paged_prefill(*(x.to(DEV) for x in args), scale=d ** -0.5)
    want, _, _ = oracle_pages.prefill(args[0], torch.nan_to_num(args[1].float()),
                                      torch.nan_to_num(args[2].float()), *args[3:], d ** -0.5)
    e, e0 = errors(o, want)
    say(f"case precision prompt d={d}: {e / e0:.4f}")
    assert e <= 1.05 * np.sqrt(2.0) * e0


@pytest.mark.parametrize("d", [64, 128, 256])
def test_shared_prefixes_lose_little(gpu_lib, d):
    args = sha.make(d + 2, [9, 12], [1100, 700], list(range(1, 22)), 2, 8, 2, d, 32, BF16)
    o = gpu_lib.gdn_paged_shared_decode(*(x.to(DEV) for x in args), scale=d ** -0.5, min_bytes=0)
    want, _, _ = oracle_pages.shared_decode(args[0], torch.nan_to_num(args[1].float()),
                                            torch.nan_to_num(args[2].float()), *args[3:], d ** -0.5)
    e, e0 = errors(o, want)
    say(f"case precision shared d={d}: {e / e0:.4f}")
    assert e <= 1.05 * np.sqrt(2.0) * e0
