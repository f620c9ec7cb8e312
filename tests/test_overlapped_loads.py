"""Kernels that are launched while the one before them still runs wait for it and then read what it wrote. A read-only
load (`__ldg`) asks for data that does not change while the kernel lives, and that wait comes after the
kernel's start: only numbers that no kernel of the library writes may be read with it (CPU only: the sources)."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "long_context_mqa_b200", "csrc")

# norm weights and the frequencies of the rotation (rope.cu)
CONSTANT = {"rope.cu": [r"__ldg\(\(const (float4|uint2)\*\)\(\(const (float|__nv_bfloat16)\*\)w \+ [ab]\)\)", r"__ldg\(inv_freq \+ i\)"]}


def read_only_loads(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    for pattern in CONSTANT.get(name, []):
        text = re.sub(pattern, "", text)
    lines = [re.sub(r"//.*", "", x) for x in text.splitlines()]
    return [x.strip() for x in lines if "__ldg(" in x or "ld.global.nc" in x]


@pytest.mark.parametrize("name", ["rope.cu", "paged_attn.cu", "pagetable.cu"])
def test_the_operators_around_the_cache_read_no_predecessors_data_as_constant(name):
    assert read_only_loads(name) == []


@pytest.mark.parametrize("name", sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu*"))))
def test_nor_does_what_reads_the_tables_and_pages_that_they_write(name):
    assert read_only_loads(name) == []
