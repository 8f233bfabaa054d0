"""Kernels that begin while the kernel before them still runs (they call wait_for_previous) must read
their inputs with ordinary loads.  The read-only path promises that nobody writes a value during the
whole kernel, which here begins before the writer of its inputs ends; and a load through a const
__restrict__ argument may be moved above the wait."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "block_causal_streaming_b200", "csrc")


def _code(path):
    """The file's text without comments."""
    with open(path) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def _overlapping():
    return sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*.cuh"))
                  if re.search(r"^\s*wait_for_previous\(\);", _code(f), re.M))


def test_the_overlapping_kernels_are_found():
    assert {"norm_rope_kernel.cuh", "fp8_block_kernel.cuh", "attn_fp8_few_kernel.cuh",
            "attn_fp8_kernel.cuh"} <= set(_overlapping())


@pytest.mark.parametrize("name", _overlapping())
def test_no_read_only_loads(name):
    code = _code(os.path.join(CSRC, name))
    for word in ("__ldg", "__restrict__", "ld.global.nc", "__ldlu", "ldg_nc"):
        assert word not in code, f"{name}: {word}"


def test_every_overlapping_kernel_waits():
    """Each kernel that is launched over the tail of another waits, and before it lets the next begin."""
    api = _code(os.path.join(CSRC, "wf_api.cu"))
    launched = set(re.findall(r"launch_early\(\s*wfk::(\w+)", api))
    assert launched
    code = "\n".join(_code(os.path.join(CSRC, f)) for f in _overlapping())
    for kernel in launched:
        body = code[re.search(r"\b%s\(" % kernel, code).end():]
        body = body[:re.search(r"^}", body, re.M).start()]
        wait = body.find("wait_for_previous();")
        assert 0 <= wait < body.find("launch_next();"), kernel
