"""Inputs and tolerances shared by the tests of the paged attention entry points.

Tolerances are derived from the roundings that the kernels make. u is half a step of the element
type relative to the value (bf16 2^-8, fp32 2^-24), w = 2^-24 that of fp32 arithmetic.
  - A score is an fp32 sum of d products: off by at most (d + 8) w times the sum S of |q_i k_i|.
    It enters an exponential whose result (hardware exp2, 1 ulp, argument rounded once) is then
    off by that much relatively, plus 4 w times the exponent's size (at most 2 S) plus 4 w.
  - A weight enters both numerator and denominator: twice its error, times the mean M of |v|
    under the weights. bf16: the numerator's weights are rounded once more, u M.
  - n summands in fp32: at most n w M in each of the two sums; rescaling and joining partial
    results multiply by rounded factors, at most one a 16-key step: counted as another n w M.
  - The output is rounded once: u |o|.
"""
import numpy as np
import torch

W32 = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def pages(g, lens, block, extra_pages=3, extra_cols=2):
    """A block table over a shuffled pool: (table int32 with -1 where unused, n_blocks)."""
    need = [-(-max(x, 0) // block) for x in lens]
    n_blocks = sum(need) + extra_pages
    ids = torch.randperm(n_blocks, generator=g).tolist()
    width = max(need + [1]) + extra_cols
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = torch.tensor(ids[at:at + k], dtype=torch.int32)
        at += k
    return table, n_blocks


def weight_error(d, n, score_sum):
    """Relative error of a softmax weight plus the error of the sums over n keys (fp32)."""
    s = np.asarray(score_sum, dtype=np.float64)[..., None]
    return 2 * ((d + 8) * W32 * s + 8 * W32 * s + 4 * W32) + 4 * n * W32


def tolerance(o, mag, score_sum, d, n, dtype):
    u = HALF_STEP[dtype]
    lost = weight_error(d, n, score_sum) + (u if dtype == torch.bfloat16 else 0.0)
    return mag * lost + u * np.abs(o) + 1e-30


def assert_within(got, want, tol, what=""):
    got = got.detach().double().cpu().numpy()
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    bad = np.abs(got - want) > tol
    if bad.any():
        i = tuple(x[0] for x in np.nonzero(bad))
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside; at {i} got {got[i]} "
                             f"want {want[i]} tolerance {tol[i] if tol.shape == got.shape else tol}")
