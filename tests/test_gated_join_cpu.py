"""A model of how the gated scan's tiles wait for each other (entering() in csrc/gated_scan.hip), run over random
interleavings on the CPU: every tile finds a known end, whatever the order in which maps and ends come out."""
import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "selective_state_space_58_amd", "csrc",
                   "gated_scan.hip")


def constants():
    m = re.search(r"constexpr int kWindow = (\d+), kHist = (\d+);", open(SRC).read())
    return int(m[1]), int(m[2])


def tile(i, maps, ends, rnd, window, hist):
    yield
    maps[i] = True
    yield
    if i == 0:   # the first tile's end comes out some time after its map
        for _ in range(rnd.randint(0, 300)):
            yield
        ends[0] = True
        return
    base = 1
    while True:
        known = []
        for j in range(window):   # the words are read at different times
            d = base + j
            known.append((ends[i - d], maps[i - d]) if d <= i else (False, False))
            if rnd.random() < 0.2:
                yield
        f = next((j for j, k in enumerate(known) if k[0]), window)
        if all(k[1] for k in known[:f]):
            if f < window:
                break
            if base + window <= i and base + 2 * window - 1 <= hist:
                base += window
        yield
    ends[i] = True


@pytest.mark.parametrize("n", [2, 16, 17, 18, 32, 33, 34, 64, 65, 66, 130])
def test_every_wait_ends(n):
    window, hist = constants()
    for seed in range(4):
        rnd = random.Random(seed)
        maps, ends = [False] * n, [False] * n
        live = {i: tile(i, maps, ends, rnd, window, hist) for i in range(n)}
        steps = 0
        while live:
            i = rnd.choice(list(live))
            try:
                next(live[i])
            except StopIteration:
                del live[i]
            steps += 1
            assert steps < 400000, "tiles %s wait for ever" % sorted(live)[:5]
        assert all(ends)
