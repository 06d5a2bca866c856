"""CPU model of the paged decode kernels' work split: the chunks of all (request, head group)
units laid end to end, each unit followed by `extra` chunks that count for the cut only, and cut
into equal runs, one per worker. The model restates the index arithmetic of the kernels and
checks that
  - every chunk of every unit is worked on once, by runs that differ in length by one chunk at
    most;
  - a unit that several workers touch has a part from each worker between the first and the last,
    each in a slot of its own, which are the slots that the join reads;
  - each unit's note is written by exactly one worker (per unit), or each worker leaves at most
    one note (per worker), and no note is left unwritten;
  - the division by multiplication is exact below 2^31.
"""
import random

import pytest

MAX_WORKERS = 1024


def cut_of(total, workers):
    n = min(total, workers)
    return (n, total // n, total % n) if n else (0, 0, 0)


def start(cut, w):
    return w * cut[1] + min(w, cut[2])


def owner(cut, x):
    n, each, more = cut
    big = more * (each + 1)
    return x // (each + 1) if x < big else more + (x - big) // each


def locate(chunks, units, extra, pos):
    """(request, first chunk of the request) that chunk `pos` lies in."""
    base = 0
    for b, n in enumerate(chunks):
        span = (n + extra) * units if n else 0
        if pos < base + span:
            return b, base
        base += span
    raise AssertionError


def run_worker(chunks, units, extra, cut, w):
    """Pieces (request, unit, c0, c1, slot, late, last worker) in the order of the kernel's loop."""
    pieces = []
    if w >= cut[0]:
        return pieces
    pos, end = start(cut, w), start(cut, w + 1)
    first = pos
    b, base = locate(chunks, units, extra, pos)

    def advance(to, request_end):
        nonlocal pos, b, base
        pos = to
        if pos < end and pos == request_end:
            base = pos
            b += 1
            while b + 1 < len(chunks) and chunks[b] == 0:
                b += 1

    while pos < end:
        n = chunks[b]
        assert n > 0
        unit, c0 = divmod(pos - base, n + extra)
        next_unit = base + (unit + 1) * (n + extra)
        request_end = base + units * (n + extra)
        if c0 >= n:
            advance(next_unit, request_end)
            continue
        c1 = min(n, c0 + end - pos)
        late = pos != first
        pieces.append((b, unit, c0, c1, 2 * w + late, late, owner(cut, pos + n - 1)))
        advance(next_unit if c1 == n else pos + c1 - c0, request_end)
    return pieces


def check(chunks, units, extra, workers):
    total = sum((n + extra) * units for n in chunks if n)
    cut = cut_of(total, workers)
    if cut[0]:
        lengths = {start(cut, w + 1) - start(cut, w) for w in range(cut[0])}
        assert max(lengths) - min(lengths) <= 1 and start(cut, cut[0]) == total
    done, parts, notes, slots = {}, {}, {}, set()
    for w in range(workers):
        unfinished = 0
        for b, unit, c0, c1, slot, late, last in run_worker(chunks, units, extra, cut, w):
            assert 0 <= unit < units
            for c in range(c0, c1):
                assert (b, unit, c) not in done
                done[b, unit, c] = w
            if c0 == 0:
                assert (b, unit) not in notes
                notes[b, unit] = (w, late, last) if c1 < chunks[b] else None
                unfinished += c1 < chunks[b]
            if not (c0 == 0 and c1 == chunks[b]):
                assert slot not in slots and 0 <= slot < 2 * workers
                slots.add(slot)
                parts.setdefault((b, unit), {})[w] = slot
        assert unfinished <= 1  # a note per worker is enough
    assert len(done) == sum(chunks) * units
    for b, n in enumerate(chunks):
        for unit in range(units if n else 0):
            note = notes[b, unit]
            if note is None:
                assert (b, unit) not in parts
                continue
            w0, late, w1 = note
            assert w1 - w0 + 1 <= MAX_WORKERS
            # part i of the join: worker w0 + i, its first slot but for a late first part
            read = {w0 + i: 2 * (w0 + i) + (late if i == 0 else 0) for i in range(w1 - w0 + 1)}
            assert read == parts[b, unit]


@pytest.mark.parametrize("extra", [0, 2, 6])
@pytest.mark.parametrize("units", [1, 3, 8])
@pytest.mark.parametrize("workers", [8, 64, 256])
def test_every_chunk_once_and_every_part_found(extra, units, workers):
    rng = random.Random(extra * 1000 + units * 10 + workers)
    cases = [[1], [0, 0, 1], [1, 0, 0], [5000], [0], [], [1] * 300, [2, 0] * 40 + [900]]
    for _ in range(25):
        n = rng.randint(1, 40)
        cases.append([rng.choice([0, 1, 2, rng.randint(1, 60), rng.randint(1, 400)])
                      for _ in range(n)])
    for chunks in cases:
        check(chunks, units, extra, workers)


def fast_div(d):
    s = 0
    while (1 << s) < d:
        s += 1
    mul = (((((1 << s) - d) << 32) // d) + 1) & 0xffffffff
    return lambda n: (((n * mul) >> 32) + n & 0xffffffff) >> s


def test_division_by_multiplication_is_exact():
    rng = random.Random(1)
    divisors = list(range(1, 700)) + [2 ** k + e for k in range(9, 31) for e in (-1, 0, 1)]
    for d in divisors:
        div = fast_div(d)
        for n in [0, 1, d - 1, d, d + 1, 2 * d - 1, 2 ** 31 - 1, (2 ** 31 - 1) // d * d,
                  (2 ** 31 - 1) // d * d - 1] + [rng.randrange(2 ** 31) for _ in range(20)]:
            if 0 <= n < 2 ** 31:
                assert div(n) == n // d, (n, d)
