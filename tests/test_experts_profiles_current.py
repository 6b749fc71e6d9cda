"""The summaries in profiles/experts describe the routed experts' kernels as they are: each
names the sha256 of the kernel source that it was captured on, which must be its present one."""
import hashlib
import os

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "roofline_driven_optimisation_gb300", "csrc")
EXPERTS = os.path.join(ROOT, "profiles", "experts")

SOURCES = {
    "blocks_kernel_swiglu_decode_64.md": "fp8_blocks.cu",
    "blocks_wide_kernel_8192.md": "fp8_blocks_wide.cu",
    "blocks_wide_kernel_swiglu_16384.md": "fp8_blocks_wide.cu",
    "quantise_rows_kernel_16384.md": "fp8_quantise.cu",
    "route_kernel_16384x256.md": "route.cu",
}


def test_every_summary_is_listed():
    assert {f for f in os.listdir(EXPERTS) if f.endswith(".md")} == set(SOURCES)


@pytest.mark.parametrize("summary", sorted(SOURCES))
def test_summary_names_the_current_source(summary):
    with open(os.path.join(EXPERTS, summary), encoding="utf-8") as f:
        text = f.read()
    with open(os.path.join(CSRC, SOURCES[summary]), "rb") as f:
        now = hashlib.sha256(f.read()).hexdigest()
    assert now in text, f"{summary} was captured on another {SOURCES[summary]} (current sha256 {now})"
