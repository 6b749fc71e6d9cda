"""The plan of routing calls on the CPU (csrc/plan.h, compiled with g++ into a small query
program): every token has a block, no more blocks than SMs, and the workspace that is measured
for a whole GB300 is enough for fewer SMs."""
import os
import random
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "roofline_driven_optimisation_gb300", "csrc")
OUT = os.path.join(ROOT, "roofline_driven_optimisation_gb300", "_build", "route_check")


@pytest.fixture(scope="module")
def plan():
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    os.makedirs(os.path.dirname(OUT), exist_ok=True)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC,
                    os.path.join(ROOT, "tests", "route_check.cpp"), "-o", OUT], check=True)

    def ask(queries):
        text = "".join(" ".join(str(x) for x in q) + "\n" for q in queries)
        r = subprocess.run([OUT], input=text, capture_output=True, text=True, check=True)
        return [tuple(int(x) for x in line.split()) for line in r.stdout.split("\n")[:len(queries)]]
    return ask


def test_plans(plan):
    got = plan([(1, 64, 152), (16, 256, 152), (17, 256, 152), (64, 256, 152), (16384, 256, 152), (16384, 256, 148),
                (16384, 1024, 148), (16384, 256, 1)])
    assert got == [(8, 1, 1, 1), (16, 1, 16, 1), (8, 3, 6, 1), (8, 8, 8, 1), (32, 152, 108, 0), (32, 148, 111, 0),
                   (8, 148, 111, 0), (32, 1, 16384, 0)]


def test_every_token_has_a_block(plan):
    rng = random.Random(0)
    tokens = [int(2 ** rng.uniform(0, 31)) for _ in range(3000)] + [2 ** 31 - d for d in range(1, 200)]
    queries = [(max(1, t), rng.choice([1, 60, 256, 257, 1024]), rng.choice([1, 2, 20, 76, 132, 148, 152, 160])) for t in tokens]
    whole = plan([(t, e, 152) for t, e, _ in queries])
    for (t, e, sms), (warps, blocks, chunk, few), (_, most, _, _) in zip(queries, plan(queries), whole):
        assert 1 <= blocks <= min(sms, 152) and chunk >= 1
        assert (blocks - 1) * chunk < t <= blocks * chunk
        assert warps in (8, 16, 32) and (warps < 32 or e <= 256) and few == (t <= 256)
        assert blocks <= most
