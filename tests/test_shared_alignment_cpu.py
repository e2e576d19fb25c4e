"""Shared memory that a kernel accesses in wider pieces than its element type is declared
with an alignment that allows it (a misaligned access faults the GPU).  Reads the kernel
sources.  CPU only."""

import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(glob.glob(os.path.join(ROOT, "rmsnorm_fwd_bwd_03_gb300", "csrc", "*.cu*")))
SIZE = {"float": 4, "uint32_t": 4, "int32_t": 4, "float2": 8, "uint2": 8, "uint64_t": 8, "double": 8, "float4": 16, "uint4": 16,
        "unsigned char": 1}

DECLARED = re.compile(r"__shared__\s+(?:__align__\((\d+)\)\s+)?([a-z_0-9]+(?: char)?)\s+(\w+)\s*\[")


def _wide_uses(text):
    """(array, bytes per access, bytes its declaration is aligned to) of every access of a
    __shared__ array through a pointer to a wider type."""
    out = []
    for use in re.finditer(r"reinterpret_cast<(?:const )?(\w+)\s*\*>\(&?(\w+)", text):
        before = [d for d in DECLARED.findall(text[:use.start()]) if d[2] == use[2]]
        if before:  # the nearest declaration above
            align, kind, name = before[-1]
            out.append((name, SIZE.get(use[1], 1), max(int(align or 0), SIZE[kind])))
    return out


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_wide_accesses_of_shared_arrays_are_aligned(path):
    with open(path, encoding="utf-8") as f:
        uses = _wide_uses(f.read())
    assert all(have >= need for _, need, have in uses), uses


def test_the_reading_sees_such_accesses():
    bad = "__shared__ float s[8];\n*reinterpret_cast<float2*>(&s[i]) = v;"
    assert _wide_uses(bad) == [("s", 8, 4)]
    assert _wide_uses(bad.replace("float s", "__align__(16) float s")) == [("s", 8, 16)]
