"""The summaries in profiles/serving describe the serving kernels as they are: each names
the sha256 of the kernel source that it was captured on, which must be its present one."""
import hashlib
import os

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "roofline_driven_optimisation_gb300", "csrc")
SERVING = os.path.join(ROOT, "profiles", "serving")

SOURCES = {
    "kv_append_pages_kernel_16384_e4m3.md": "kv_append.cu",
    "kv_attention_kernel_16x4096_int8.md": "kv_attention.cu",
    "sample_stream_kernel_384x131071_fp32.md": "sample.cu",
}


def test_every_summary_is_listed():
    assert {f for f in os.listdir(SERVING) if f.endswith(".md")} == set(SOURCES)


@pytest.mark.parametrize("summary", sorted(SOURCES))
def test_summary_names_the_current_source(summary):
    with open(os.path.join(SERVING, summary), encoding="utf-8") as f:
        text = f.read()
    with open(os.path.join(CSRC, SOURCES[summary]), "rb") as f:
        now = hashlib.sha256(f.read()).hexdigest()
    assert now in text, f"{summary} was captured on another {SOURCES[summary]} (current sha256 {now})"
