"""A thread's walk over the values of a page's rows (csrc/row_walk.cuh), compiled for the
host: every place once, also where the rows hold more than 2^31 values."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "roofline_driven_optimisation_gb300", "csrc")
OUT = os.path.join(ROOT, "roofline_driven_optimisation_gb300", "_build", "rw_check")


@pytest.fixture(scope="module")
def walk():
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    os.makedirs(os.path.dirname(OUT), exist_ok=True)
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-I", CSRC,
                    os.path.join(ROOT, "tests", "rw_check.cpp"), "-o", OUT], check=True)

    def ask(*numbers):
        r = subprocess.run([OUT], input=" ".join(map(str, numbers)) + "\n", capture_output=True, text=True, check=True)
        return [int(x) for x in r.stdout.split()]
    return ask


@pytest.mark.parametrize("width", [1, 2, 3, 40, 127, 128, 129, 512])
@pytest.mark.parametrize("rows", [0, 1, 2, 17, 256])
def test_every_place_once(walk, width, rows):
    for first in (0, 1, 63, 127):
        places = range(first, width * rows, 128)
        n, row, at, same = walk(first, 128, width, rows)
        assert n == len(places) and same == 1
        if n:
            assert (row, at) == divmod(places[-1], width)


@pytest.mark.parametrize("width,rows", [(512, 2 ** 23), (192, 2 ** 24 + 7), (1, 2 ** 31 - 1)])
def test_more_than_32_bits_of_values(walk, width, rows):
    for first in (0, 127):
        places = range(first, width * rows, 128)
        assert walk(first, 128, width, rows) == [len(places), *divmod(places[-1], width), 1]
