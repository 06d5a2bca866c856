"""CPU model of the tile schedule of the latent prefill's attend kernel: two LDS buffers of keys
and two of values, the next tile's scores formed beside a tile's softmax, one barrier a tile. A
wave's rows may end before the workgroup's last tile. The tile whose scores a step forms is read
from the kernel's source; the model checks that
  - no wave reads a buffer that is being filled between the same two barriers, or one whose fill
    has not been waited for;
  - the scores and values that are used are those of the right tile.
"""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "gated_delta_rule_prefill_amd", "csrc", "latent_prefill.hip")


def scored_tile():
    """The source's expression for it, as a function of t, mine and nt."""
    text = open(SOURCE, encoding="utf-8").read()
    (expr,) = re.findall(r"scores\(([^,\[]+), next,", text)
    m = re.fullmatch(r"(.+?)\?(.+?):(.+)", expr)
    expr = f"({m[2].strip()}) if ({m[1].strip()}) else ({m[3].strip()})" if m else expr
    return lambda t, mine, nt: eval(expr, {"__builtins__": {}}, dict(t=t, mine=mine, nt=nt))


def check(nt, mine, tile_of):
    keys, values = [None, None], [None, None]        # tile that a buffer holds
    filling_k, filling_v = {0: 0}, {}                # buffer -> tile, since the last wait

    def wait():
        for held, filling in ((keys, filling_k), (values, filling_v)):
            for buf, tile in filling.items():
                held[buf] = tile
            filling.clear()

    wait()                                           # load_keys(0), waited for, barrier
    if nt > 1:
        filling_k[1] = 1
    filling_v[0] = 0
    scored = None
    if mine > 0:
        assert keys[0] == 0 and 0 not in filling_k
        scored = 0
    for t in range(nt):
        wait()
        if t + 2 < nt:
            filling_k[t & 1] = t + 2
        if t + 1 < nt:
            filling_v[(t + 1) & 1] = t + 1
        if t >= mine:
            continue
        assert scored == t
        tile = tile_of(t, mine, nt)
        buf = tile & 1
        assert buf not in filling_k, f"tile {t} of {nt}: reads a key buffer that is being filled"
        scored = tile if keys[buf] == tile else None  # (not used behind the wave's last tile)
        assert (t & 1) not in filling_v and values[t & 1] == t
    assert mine <= nt


@pytest.mark.parametrize("nt", range(1, 9))
def test_no_buffer_is_read_while_it_is_filled(nt):
    tile_of = scored_tile()
    for mine in range(nt + 1):
        check(nt, mine, tile_of)
