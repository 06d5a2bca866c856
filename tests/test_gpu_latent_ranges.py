"""The latent forms over the range of their bf16 inputs: latents, weights and queries far from 1, in
tiles of 64 keys that differ by many powers of two. gdn_latent_prefill has to scale its fp16 keys,
values and weights for them, gdn_latent_decode the 4-bit rests of its absorbed queries."""
import pytest
import torch

import test_gpu_latent as lat
from gpu_util import say

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
CTX, NEW = [150, 0, 300], [120, 70, 9]


def _case(seed, R, d, H):
    case = list(lat._prefill_case(seed, CTX, NEW, H, R, d, 16, poison=False))
    return case, [c + n for c, n in zip(CTX, NEW)]


def _rows(table, i, lo, hi):
    j = torch.arange(lo, hi)
    return table[i][j // 16].long(), j % 16


@pytest.mark.parametrize("R,d", [(512, 128), (256, 64)])
@pytest.mark.parametrize("powers", [[0, 20, -20, 40, -40, 9], [-45, -45, -45, 0, 50, 50],
                                    [60, 60, 60, 60, 60, 60], [7, 8, 9, 7, 8, 9], [-9, -10, -11, -9, -12, -8]])
def test_latents_of_any_size(R, d, powers):
    """Tiles of a request whose latents differ: weights come from the rotary keys, so that every
    tile counts; rows before a tile of large latents see small ones only."""
    say(f"case ranges latents R={R} {powers}")
    case, lens = _case(1, R, d, 2)
    for i, n in enumerate(lens):
        for t in range(0, n, 64):
            rows = _rows(case[4], i, t, min(t + 64, n))
            case[3][rows[0], rows[1], :R] *= 2.0 ** powers[(t // 64 + i) % len(powers)]
    case[0].zero_()
    lat._check_prefill(tuple(case), every=4)


@pytest.mark.parametrize("powers", [[20, 0, 0, 0, 0, 0], [0, 50, 0, 0, 0, 0], [-30, 30, -30, 0, 0, 0],
                                    [0, 60, -40, 60, -40, 0], [12, 0, 12, 0, 12, 0]])
def test_tiles_of_large_latents_that_no_query_looks_at(powers):
    """Their weights are 2^-100 or less of the others': outputs are those of the small tiles."""
    say(f"case ranges ignored {powers}")
    R = 512
    case, lens = _case(11, R, 128, 2)
    for i, n in enumerate(lens):
        for t in range(0, n, 64):
            rows = _rows(case[4], i, t, min(t + 64, n))
            p = powers[(t // 64) % len(powers)]
            case[3][rows[0], rows[1], :R] *= 2.0 ** p
            case[3][rows[0], rows[1], R] = 0.0 if p <= min(powers) else -1500.0
    case[0].zero_()
    case[1][..., 0] = 1.0
    lat._check_prefill(tuple(case), every=3)


@pytest.mark.parametrize("power", [30, -30, 12])
def test_weights_and_queries_of_any_size(power):
    """Heads whose key weights and queries differ by powers of two that cancel, value weights
    that do not."""
    say(f"case ranges weights 2^{power}")
    R, d, H = 512, 64, 4
    case, _ = _case(2, R, d, H)
    for h in range(H):
        case[2][h, :d] *= 2.0 ** (power * (h - 1))
        case[0][:, h] *= 2.0 ** (-power * (h - 1))
        case[2][h, d:] *= 2.0 ** (power * (2 - h))
    lat._check_prefill(tuple(case), every=4)


@pytest.mark.parametrize("power", [50, -50])
def test_scales_that_cancel_the_queries(power):
    say(f"case ranges queries 2^{power}")
    case, _ = _case(3, 256, 128, 2)
    case[0] *= 2.0 ** power
    case[1] *= 2.0 ** power
    case[7] *= 2.0 ** -power
    lat._check_prefill(tuple(case), every=4)


@pytest.mark.parametrize("power", [-60, -100, 0])
def test_key_weights_that_vanish(power):
    """Scores of the rotary keys alone, beside queries of any size."""
    say(f"case ranges vanishing weights 2^{power}")
    for weights in (0.0, 2.0 ** -100):
        case, _ = _case(12, 256, 64, 2)
        case[2][:, :64] *= weights
        case[0] *= 2.0 ** power
        lat._check_prefill(tuple(case), every=4)


def test_zeros():
    """No latent, no weight or no query that could say how large the others may be."""
    say("case ranges zeros")
    for at in (0, 1, 2, 3):
        case, _ = _case(4 + at, 256, 64, 2)
        case[at] = torch.zeros_like(case[at])
        if at in (2, 3):
            o = lat._run_prefill(tuple(case))
            assert not o.any()
        else:
            lat._check_prefill(tuple(case), every=4)


@pytest.mark.parametrize("value", [float("inf"), 3e38, float("nan")])
def test_one_requests_rows_do_not_reach_the_others(value):
    """Requests share workgroups of the expanding launch; an absent key stands for any row."""
    say(f"case ranges foreign {value}")
    case, lens = _case(9, 512, 128, 2)
    want = lat._run_prefill(tuple(case))
    rows = _rows(case[4], 1, 0, lens[1])
    bad = list(case)
    bad[3] = case[3].clone()
    bad[3][rows[0], rows[1]] = value
    # and the row that absent keys read
    owner = [int(i) for i in range(3) if (case[4][i] == 0).any()]
    if owner != [1]:
        swap = int(case[4][1, 0])
        moved = bad[3].clone()
        moved[0], moved[swap] = bad[3][swap], bad[3][0]
        table = case[4].clone()
        table[case[4] == 0], table[case[4] == swap] = swap, 0
        bad[3], bad[4] = moved, table
    got = lat._run_prefill(tuple(bad))
    keep = torch.ones(got.shape[0], dtype=torch.bool)
    keep[NEW[0]:NEW[0] + NEW[1]] = False
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_bad_weight_spoils_its_own_dim_only(value):
    say(f"case ranges weight {value}")
    d = 64
    case, _ = _case(10, 512, d, 3)
    want = lat._run_prefill(tuple(case))
    case[2] = case[2].clone()
    case[2][1, d + 5, 77] = value
    got = lat._run_prefill(tuple(case))
    keep = torch.ones(3, d, dtype=torch.bool)
    keep[1, 5] = False
    assert torch.equal(got[:, keep], want[:, keep])
    assert not torch.isfinite(got[:, 1, 5].float()).any()


# ---------------------------------------------------------------------------------- decode
def _decode(seed, R, d, H, P):
    return list(lat._decode_case(seed, [130, 70, 0, 5], P, H, R, d, 16, poison=False))


@pytest.mark.parametrize("R,d,H,P", [(512, 128, 3, 1), (256, 64, 20, 2), (512, 64, 40, 2)])
@pytest.mark.parametrize("power", [60, -60, -110])
def test_decode_queries_of_any_size(R, d, H, P, power):
    say(f"case ranges decode queries R={R} 2^{power}")
    case = _decode(20, R, d, H, P)
    case[0] *= 2.0 ** power
    case[1] *= 2.0 ** power
    case[6] *= 2.0 ** -power
    lat._check_decode(tuple(case))


@pytest.mark.parametrize("power", [20, -20, 6])
def test_decode_columns_of_any_size(power):
    """Columns of the latents and of the weights that differ by powers of two that cancel: every
    absorbed query's number counts, the small ones beside the large."""
    say(f"case ranges decode columns 2^{power}")
    case = _decode(21, 512, 128, 20, 1)
    for at in (slice(0, 40), slice(130, 131), slice(300, 420)):
        case[2][:, :128, at] *= 2.0 ** power
        case[3][..., at] *= 2.0 ** -power
    case[2][:, 128:] *= 2.0 ** -abs(power)     # (the values are not what is looked at)
    lat._check_decode(tuple(case))


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_decode_bad_numbers_stay_in_their_row(value):
    say(f"case ranges decode {value}")
    case = _decode(22, 512, 128, 20, 2)
    want = lat._run_decode(tuple(case))
    bad = list(case)
    bad[0] = case[0].clone()
    bad[0][1, 1, 7, 5] = value
    bad[0][0, 0, 3] = 0.0
    got = lat._run_decode(tuple(bad))
    keep = torch.ones(got.shape[:3], dtype=torch.bool)
    keep[1, 1, 7] = keep[0, 0, 3] = False
    assert torch.equal(got[keep], want[keep])
    assert not torch.isfinite(got[1, 1, 7].float()).any()
    assert torch.isfinite(got[0, 0, 3].float()).all()
