"""Host-side checks of the counts and walks that the block-scaled and experts' kernels use, at
sizes up to 2^31 - 1: `extents_check.cpp` compares dense_gemm_06_amd/csrc/extents.h with
64-bit arithmetic, under the undefined-behaviour sanitizer. No GPU is involved."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_extents(tmp_path):
    exe = tmp_path / "extents_check"
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                        os.path.join(ROOT, "tests", "extents_check.cpp"), "-o", str(exe)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "0 failures" in r.stdout, (r.stdout[-2000:], r.stderr[-2000:])


def source(name):
    """A kernels' source without its comments."""
    return re.sub(r"//[^\n]*", "", open(os.path.join(ROOT, "dense_gemm_06_amd", "csrc", name)).read())


def test_products_count_through_extents():
    """`(size + 127) / 128` wraps near 2^31, pieces<128>(size) does not."""
    assert not re.findall(r"\((?:g\.[MNK]|hi - lo) \+ \w+ - 1\) / ", source("kernel_block.h"))
    assert not re.findall(r"\(a\.tokens \+ \w+ - 1\) / ", source("route.hip"))


def test_experts_tiles_are_capped():
    """Offsets that do not grow make ranges overlap, and their tiles' sum pass 2^31."""
    assert not re.findall(r"total \+= ", source("kernel_block.h"))


# kernels whose loops over sizes up to 2^31 go by steps of the grid, of the workgroup or of a wave
WALKS = ["kernel_block.h", "combine.hip", "route.hip"]


@pytest.mark.parametrize("name", WALKS)
def test_kernels_walk_through_extents(name):
    """A 32-bit counter wraps past an end within one step of 2^31 and reads or writes out of range."""
    size = r"(?:a\.(?:tokens|cols|capacity|n)|g\.[MNKE])\b|start\["
    assert not re.findall(r"for \(int \w+ = [^;]*;[^;]*(?:%s)[^;]*; \w+ \+=" % size, source(name))
    assert not re.findall(r"\w+ \+ \d{2,} <= (?:%s)" % size, source(name))  # `at + 2048 <= size` wraps too
