"""Which operands the kernels may read through the read-only path (`__ldg`, `const __restrict__`
parameters): weights alone. A kernel begins before the previous one on its stream has ended
(programmatic dependent launch), so everything that an earlier call may have written is
written during its life, and is read by ordinary loads after its wait. CPU only: the sources are
read as text."""
import os
import re

import pytest

from quantized_weight_matmul_q4_gb300.build import CSRC

# Pointers to weights, their scales and zero points, by their names in the kernels.
WEIGHTS = {"W", "scales", "zeros", "w4"}
FILES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", FILES)
def test_loads_past_the_ordinary_path(name):
    for m in re.finditer(r"__ldg\(\s*(?:reinterpret_cast<[^>]*>\()?\s*(?:a\.|p\.)?(\w+)", _source(name)):
        assert m.group(1) in WEIGHTS, f"{name}: {m.group(0)}"
    assert "ld.global.nc" not in _source(name)


@pytest.mark.parametrize("name", FILES)
def test_read_only_parameters_of_kernels(name):
    for kernel in re.finditer(r"__global__.*?\((.*?)\)\s*\{", _source(name), re.S):
        for m in re.finditer(r"const\s+\w+\s*\*\s*__restrict__\s+(\w+)", kernel.group(1)):
            assert m.group(1) in WEIGHTS, f"{name}: {m.group(0)}"
