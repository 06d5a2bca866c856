"""CPU model of the step schedule of paged_attend.h: key and value tiles in two or three LDS buffers
each, loaded ahead; the cache rows of a step's keys, put down by the waves in turns from table
entries asked for a step before, in eight slots; one barrier a step. How far ahead each of these
runs is read from the source. The model checks for runs of any length that
  - a wave reads keys, values and rows of the right step, whose loads or stores were waited for
    before the last barrier;
  - no buffer or slot is written between the same two barriers in which it is read;
  - a wave puts down the table entry that it asked for, in the step after.
"""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "gated_delta_rule_prefill_amd", "csrc", "paged_attend.h")


def ahead():
    """Steps ahead of c, from the source's step and prologue: functions of LEAD."""
    text = open(SOURCE, encoding="utf-8").read()
    step = text[text.index("auto step = [&]"):text.index("if (c1 > c0) {")]
    start = text[text.index("if (c1 > c0) {"):text.index("for (int c = c0; c < c1; c += 2)")]

    def one(part, pattern, which=0):
        found = re.findall(pattern, part)
        expr = found[which]
        return lambda lead, name="LEAD": eval(expr, {"__builtins__": {}}, {"LEAD": lead, "c": 0,
                                                                         "c0": 0})
    return dict(
        load_k=one(step, r"load_keys\(([^)]+)\)"), load_v=one(step, r"load_values\(([^)]+)\)"),
        late_k=one(step, r"!ROWS_EARLY\) rows_of\(([^,]+), k_rows"),
        late_v=one(step, r"!ROWS_EARLY\) rows_of\(([^,]+), v_rows"),
        rows_k=one(step, r"(?<!\) )rows_of\(([^,]+), k_rows"),
        rows_v=one(step, r"(?<!\) )rows_of\(([^,]+), v_rows"),
        put=one(step, r"put_rows\(([^,]+), page"), ask=one(step, r"page_of\(([^)]+)\)"),
        first_rows=one(start, r"i < ([^;]+); i \+= X::WAVES\) put_rows"),
        first_ask=one(start, r"page = page_of\(([^)]+)\)"),
        next_k=one(start, r"if \([^)]*\) load_keys\(([^)]+)\)", -1),
        early_k=one(start, r"rows_of\(([^,]+), k_rows\)", -1),
        early_v=one(start, r"rows_of\(([^,]+), v_rows\)", -1))


class Store:
    """Numbered places: what each holds for everyone, and what is written since the last barrier."""

    def __init__(self, n):
        self.held, self.fresh, self.read = [None] * n, {}, set()

    def write(self, step):
        at = step % len(self.held)
        assert at not in self.read and at not in self.fresh, f"step {step} overwrites what is in use"
        self.fresh[at] = step

    def get(self, step):
        at = step % len(self.held)
        assert at not in self.fresh, f"step {step} is read while its place is written"
        self.read.add(at)
        return self.held[at]

    def barrier(self):
        for at, step in self.fresh.items():
            self.held[at] = step
        self.fresh, self.read = {}, set()


def run(a, lead, early, waves, c0, c1, mine):
    """One unit's steps; mine[w]: the step behind wave w's last one."""
    keys, values, rows = Store(2 + lead), Store(2 + lead), Store(8)
    page = [None] * waves                    # step whose table entry a wave holds

    def load(tiles, step, held):
        assert held == step, f"tile {step} loaded with the rows of {held}"
        tiles.write(step)

    def barrier():
        for s in (keys, values, rows):
            s.barrier()
    for i in range(a["first_rows"](lead)):
        rows.write(c0 + i)
    barrier()
    load(keys, c0, rows.get(c0))
    if lead and c0 + 1 < c1:
        load(keys, c0 + 1, rows.get(c0 + 1))
    barrier()
    if c0 + a["first_ask"](lead) < c1:
        page[c0 & (waves - 1)] = c0 + a["first_ask"](lead)
    n = c0 + a["next_k"](lead)
    if n < c1:
        load(keys, n, rows.get(n))
    load(values, c0, rows.get(c0))
    if lead and c0 + 1 < c1:
        load(values, c0 + 1, rows.get(c0 + 1))
    k_rows, v_rows = (rows.get(c0 + a[x](lead)) for x in ("early_k", "early_v"))
    for w in range(waves):
        if c0 < mine[w]:
            assert keys.get(c0) == c0
            if lead:
                keys.get(c0 + 1)
    for c in range(c0, c1):
        barrier()                            # all loads were waited for
        k, v = c + a["load_k"](lead), c + a["load_v"](lead)
        if k < c1:
            load(keys, k, k_rows if early else rows.get(c + a["late_k"](lead)))
        if v < c1:
            load(values, v, v_rows if early else rows.get(c + a["late_v"](lead)))
        if early:
            k_rows, v_rows = (rows.get(c + a[x](lead)) for x in ("rows_k", "rows_v"))
        w, x = c & (waves - 1), c + a["put"](lead)
        if x < c1:
            assert page[w] == x, f"wave {w} puts down step {x}, holds {page[w]}"
            rows.write(x)
        w, x = (c + 1) & (waves - 1), c + a["ask"](lead)
        if x < c1:
            page[w] = x
        for w in range(waves):
            if c >= mine[w]:
                continue
            assert values.get(c) == c
            if c + 1 < mine[w]:              # (scores behind a wave's last step are not used)
                assert keys.get(c + 1) == c + 1
                assert rows.get(c + 1) == c + 1
            else:
                keys.get(c + 1)
            if lead and c + 2 < mine[w]:
                assert keys.get(c + 2) == c + 2


def test_the_source_is_understood():
    a = ahead()
    assert all(isinstance(f(0), int) and f(1) >= f(0) for f in a.values())


@pytest.mark.parametrize("lead,early,waves", [(1, True, 8), (0, True, 8), (0, False, 8), (0, False, 4)])
def test_runs_of_any_length(lead, early, waves):
    a = ahead()
    for c0 in (0, 1, 3, 7, 250):
        for steps in range(1, 30):
            c1 = c0 + steps
            run(a, lead, early, waves, c0, c1, [c1] * waves)
            run(a, lead, early, waves, c0, c1,
                [min(c1, c0 + (5 * w + steps) % (steps + 2)) for w in range(waves)])


@pytest.mark.parametrize("name", ["load_k", "load_v", "rows_k", "put", "ask", "first_rows"])
def test_the_model_notices_another_distance(name):
    a = ahead()
    right = a[name]
    for off in (-1, 1):
        a[name] = lambda lead: right(lead) + off
        if name == "first_rows" and off == 1:
            continue                         # one row more than is needed does no harm
        with pytest.raises(AssertionError):
            run(a, 1, True, 8, 0, 25, [25] * 8)
