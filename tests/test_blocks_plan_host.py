"""The plan of block-scaled products on the CPU: row tiles and splits of K of csrc/plan.h,
compiled with g++ into a small query program."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "roofline_driven_optimisation_gb300", "csrc")
OUT = os.path.join(ROOT, "roofline_driven_optimisation_gb300", "_build", "blocks_check")
SMS = 152


@pytest.fixture(scope="module")
def plan():
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    os.makedirs(os.path.dirname(OUT), exist_ok=True)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC,
                    os.path.join(ROOT, "tests", "blocks_check.cpp"), "-o", OUT], check=True)

    def ask(queries):
        text = "".join(" ".join(str(int(x)) for x in q) + "\n" for q in queries)
        r = subprocess.run([OUT], input=text, capture_output=True, text=True, check=True)
        return [tuple(int(x) for x in line.split()) for line in r.stdout.split("\n")[:len(queries)]]
    return ask


def test_choices(plan):
    #          rows, experts, N, blocks of K, two weights
    cases = {(1, 1, 11008, 32, 0): (32, 3), (1, 1, 128, 32, 0): (32, 8), (1, 1, 128, 3, 0): (32, 1),
             (64, 1, 4096, 86, 0): (64, 4), (64, 1, 11008, 32, 0): (64, 1), (192, 1, 11008, 32, 0): (256, 1), (8192, 1, 11008, 32, 0): (256, 1),
             # routed: 8 experts of a row each, gate and up; 64 experts of 6 rows; of 1536
             (8, 64, 1408, 16, 1): (32, 3), (384, 64, 1408, 16, 1): (32, 1), (4096, 64, 1408, 16, 1): (32, 1), (6144, 64, 1408, 16, 1): (256, 1), (98304, 64, 1408, 16, 1): (256, 1)}
    got = plan([q + (SMS, 0) for q in cases])
    assert got == list(cases.values())


def test_every_choice_can_run(plan):
    rng = random.Random(1)
    queries = [(max(1, int(2 ** rng.uniform(0, 30))), rng.choice([1, 1, 2, 8, 64, 1024]), int(2 ** rng.uniform(0, 17)),
                max(1, int(2 ** rng.uniform(0, 8))), rng.random() < 0.4, SMS, rng.choice([0, 0, 0, 128, 256]))
               for _ in range(4000)]
    for (rows, experts, N, kblocks, two, sms, forced), (nt, split) in zip(queries, plan(queries)):
        assert nt in ((32, 256) if two else (32, 64, 128, 256)) and 1 <= split <= 8
        assert split == 1 or nt <= 128 and 4 * split <= kblocks
        met = min(experts, rows)
        mean = -(-rows // met)
        tiles = -(-N // 128)
        if forced:
            assert split == 1 and nt == (32 if two and forced == 128 else forced)
        elif nt < 256:
            # every CTA of a split has an SM of its own, or half of one
            assert split == 1 or met * -(-mean // nt) * tiles * split <= (2 if nt == 32 else 1) * sms
        else:
            assert mean > (64 if two or experts > 1 else 96)
