"""CPU model of how paged_attend.h cuts the stream of all units over the workers. The number of
runs, their starts and owners are read from the source; checked are that the runs follow one
another, that none is shorter than the least that the source names, and that a position's owner is
the worker whose run it lies in."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "gated_delta_rule_prefill_amd", "csrc", "paged_attend.h")


def cut():
    """(least run, runs(total, workers), start(w, total, n), owner(x, total, n)) of the source."""
    text = open(SOURCE, encoding="utf-8").read()
    least = int(re.search(r"constexpr int ATTEND_MIN_RUN = (\d+);", text)[1])
    extra = int(re.search(r"constexpr int ATTEND_EXTRA = (\d+);", text)[1])
    body = text[text.index("struct AttendCut"):]

    def function(pattern, names):
        expr = re.sub(r"\(int\)", "", re.search(pattern, body)[1]).replace("/", "//")
        return lambda *a: eval(expr, {"__builtins__": {}},
                               dict(zip(names, a), ATTEND_MIN_RUN=least))
    n = function(r"int64_t n = ([^;]+);", ["total"])
    return (least, extra, lambda total, workers: min(n(total), workers),
            function(r"start\(int w\) const \{ return ([^;]+);", ["w", "total", "n"]),
            function(r"owner\(int64_t x\) const \{\s*return ([^;]+);", ["x", "total", "n"]))


def test_the_stream_is_cut_into_runs():
    least, extra, runs, start, owner = cut()
    assert runs(0, 256) == 0  # no units, no runs
    for total in list(range(extra, 60)) + [511, 512, 513, 600, 1023, 4097]:
        for workers in (8, 64, 256):
            n = runs(total, workers)
            assert 1 <= n <= workers
            bounds = [start(w, total, n) for w in range(n + 1)]
            assert bounds[0] == 0 and bounds[-1] == total
            sizes = [b - a for a, b in zip(bounds, bounds[1:])]
            assert min(sizes) >= least, f"a run of {min(sizes)} of {total} positions"
            assert max(sizes) - min(sizes) <= 1
            for w in range(n):
                for x in {bounds[w], bounds[w + 1] - 1}:
                    assert owner(x, total, n) == w


@pytest.mark.parametrize("total", [10 ** 6 + 1, 2 ** 40 + 12345])
def test_long_streams(total):
    least, extra, runs, start, owner = cut()
    n = runs(total, 256)
    assert n == 256
    assert all(owner(start(w, total, n), total, n) == w for w in range(n))
    assert all(owner(start(w + 1, total, n) - 1, total, n) == w for w in range(n))
