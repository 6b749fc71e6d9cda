"""The hardware barriers of the block-scaled pair kernel (csrc/fp8_blocks_wide.cu), as a model
on the CPU: a signal warp and two halves of four drain warps go through the same blocks, with
a barrier for each accumulator buffer and half.  An abort may come at any block and with the
warps anywhere; every warp has to reach the end all the same.

The model has both forms of the signal warp.  One that arrives without waiting until an abort
and waits from then on (``arrives=True``) is left hanging by some order of the warps, so the
kernel must not have that form."""
import os
import random
import re

import pytest

from conftest import ROOT

SOURCE = os.path.join(ROOT, "roofline_driven_optimisation_gb300", "csrc", "fp8_blocks_wide.cu")
WARPS, HALF = 8, 4


class Barrier:
    """bar.sync / bar.arrive with a count of five warps: the phase ends with the fifth."""

    def __init__(self):
        self.here, self.phase = 0, 0

    def arrive(self):
        phase = self.phase
        self.here += 1
        if self.here == HALF + 1:
            self.here, self.phase = 0, phase + 1
        return phase


def run(blocks, items, abort_at, seed, arrives, meet):
    """True if all warps reach the end.  The abort: the accumulator of (block, half) number
    abort_at never comes.  meet: the drain warps of both halves meet behind each item."""
    rng = random.Random(seed)
    bars = {(b, h): Barrier() for b in range(2) for h in range(2)}
    both = dict(here=0, phase=0)
    drained = [0] * WARPS                     # blocks whose buffer a warp has handed back
    gave_up = [False]

    def signal():
        n = 0
        for block in range(blocks * items):
            for h in range(2):
                # the MMA's result: its buffer was handed back by the four warps two blocks before
                while not gave_up[0] and not all(drained[4 * h + w] >= block - 1 for w in range(HALF)):
                    yield
                if n >= abort_at:
                    gave_up[0] = True
                n += 1
                bar = bars[block % 2, h]
                phase = bar.arrive()
                if not arrives or gave_up[0]:
                    while bar.phase == phase:
                        yield
                yield

    def drain(w):
        for block in range(blocks * items):
            bar = bars[block % 2, w // 4]
            phase = bar.arrive()
            while bar.phase == phase:
                yield
            drained[w] = block + 1
            yield
            if block % blocks == blocks - 1 and meet:
                phase = both["phase"]
                both["here"] += 1
                if both["here"] == WARPS:
                    both.update(here=0, phase=phase + 1)
                while both["phase"] == phase:
                    yield

    weights = [rng.choice([1, 1, 1, 20]) for _ in range(WARPS + 1)]
    live = dict(enumerate([signal()] + [drain(w) for w in range(WARPS)]))
    idle = 0
    while live:
        k = rng.choices(list(live), [weights[i] for i in live])[0]
        before = (tuple(drained), gave_up[0], both["here"], both["phase"],
                  tuple((b.here, b.phase) for b in bars.values()), len(live))
        try:
            next(live[k])
        except StopIteration:
            del live[k]
        after = (tuple(drained), gave_up[0], both["here"], both["phase"],
                 tuple((b.here, b.phase) for b in bars.values()), len(live))
        idle = 0 if after != before else idle + 1
        if idle > 4000:                       # nobody has moved for hundreds of turns each
            return False
    return True


@pytest.mark.parametrize("meet", [False, True])
@pytest.mark.parametrize("blocks,items", [(1, 1), (1, 4), (2, 3), (5, 2), (8, 1)])
def test_every_warp_reaches_the_end(blocks, items, meet):
    for abort_at in range(2 * blocks * items + 1):          # the last: no abort
        for seed in range(8):
            assert run(blocks, items, abort_at, seed, False, meet), (abort_at, seed)


def test_arrivals_ahead_of_the_drain_warps_can_hang():
    ends = [run(6, 1, abort_at, seed, True, False) for abort_at in range(2, 11) for seed in range(8)]
    assert not all(ends)
    assert all(run(6, 1, 12, seed, True, False) for seed in range(8))          # without an abort they do not


def test_the_kernel_only_waits_at_these_barriers():
    with open(SOURCE, encoding="utf-8") as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert "bar.arrive" not in code
    # five warps at 1 to 4, eight at 5
    assert sorted(set(re.findall(r"bar\.sync (\d+), (\d+)", code))) == \
        [("1", "160"), ("2", "160"), ("3", "160"), ("4", "160"), ("5", "256")]
