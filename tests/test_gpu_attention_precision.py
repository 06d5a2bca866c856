"""What the latent forms lose between their inputs and the rounding of their outputs, over all
outputs together: the 2-norm of the error against the fp64 reference, in terms of e0, that of the
reference rounded to bf16 once.

Derivation. Roundings are independent; a bf16 number's relative error is spread over the half step
alike for outputs and weights, so each rounded kind of operand that enters a sum of n products of
zero-mean values with relative errors as large as e0 moves the sum by e0 of sqrt(sum of squares),
which is at most the expected size of the sum itself. Their squares add up.
  - gdn_latent_decode rounds the softmax weights to bf16: sqrt(1 + 1) e0.
  - gdn_latent_prefill rounds keys, values and weights to 11 significant bits, an eighth of a bf16
    step each (a key's error reaches an output through its score, which scale |q| |k| / sqrt(d)
    multiplies: about twice): sqrt(1 + (1 + 1 + 4) / 64) e0.
5 % on top for the spread over the inputs drawn."""
import numpy as np
import pytest
import torch

import test_gpu_latent as lat
from gpu_util import say
from oracle import attention

pytestmark = pytest.mark.gpu


def _errors(got, want):
    """(relative 2-norm error, the same of the reference rounded to bf16)."""
    once = torch.from_numpy(want).to(torch.bfloat16).double().numpy()
    norm = np.linalg.norm(want)
    return (np.linalg.norm(got.double().cpu().numpy() - want) / norm,
            np.linalg.norm(once - want) / norm)


@pytest.mark.parametrize("R,d,H,P,lens", [
    (512, 128, 16, 1, [60, 500, 1100, 200, 900]), (256, 64, 32, 1, [60, 500, 1100, 200, 900]),
    (512, 128, 20, 1, [60, 500, 1100, 200]), (512, 64, 20, 4, [60, 500, 300]),
    (256, 128, 128, 1, [60, 500]), (512, 128, 128, 1, [60, 500])])
def test_latent_decode_loses_little(R, d, H, P, lens):
    case = lat._decode_case(R + H, lens, P, H, R, d, 16, poison=False)
    want = attention.latent_absorbed(*case[:3], case[3].double(), *case[4:])
    e, e0 = _errors(lat._run_decode(case), want)
    say(f"case precision decode R={R} d={d} H={H} P={P}: {e:.5f}, rounded once {e0:.5f}")
    assert e <= 1.05 * np.sqrt(2.0) * e0


@pytest.mark.parametrize("R,d,H,ctx,new", [
    (512, 128, 8, [0, 300], [130, 70]), (256, 64, 8, [0, 300], [130, 70]),
    (512, 64, 4, [900, 0], [40, 65]), (256, 128, 4, [900, 0], [40, 65])])
def test_latent_prefill_loses_little(R, d, H, ctx, new):
    case = lat._prefill_case(R + d, ctx, new, H, R, d, 16, poison=False)
    want = attention.latent_expanded(*case[:3], case[3].double(), *case[4:])
    e, e0 = _errors(lat._run_prefill(case), want)
    say(f"case precision prefill R={R} d={d} H={H}: {e:.5f}, rounded once {e0:.5f}")
    assert e <= 1.05 * np.sqrt(1 + 6 / 64) * e0
