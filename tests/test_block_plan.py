"""CPU tests of which kernel a block-scaled product takes: `block_plan_print.cpp` prints what
dense_gemm_06_amd/csrc/block_plan.h chooses. No GPU is involved."""
import os
import random
import shutil
import subprocess

import pytest

from block_shapes import DIRECT, EXPERTS, GRADIENT, PLAIN, SHAPES, SKINNY, STAGED, TURNED

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """A function from argument tuples to (kernel, rows, columns, slices, rest) tuples."""
    exe = str(tmp_path_factory.mktemp("plan") / "block_plan_print")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                        os.path.join(ROOT, "tests", "block_plan_print.cpp"), "-o", exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]

    def ask(asked):
        text = "\n".join(" ".join(map(str, a)) for a in asked)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-3000:]
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]

    return ask


def test_shapes_take_their_kernels(plans):
    got = plans([s.plan_arguments() for s in SHAPES])
    want = [(s.kernel, *s.tile, s.split, s.rest) for s in SHAPES]
    assert [(repr(s), g) for s, g in zip(SHAPES, got)] == [(repr(s), w) for s, w in zip(SHAPES, want)]


def test_shapes_cover_the_kernels():
    """Every kernel that a launch can name, with either kind of scales of B, in every mode that takes it."""
    have = {(s.mode, s.kernel, s.tile, s.turn, s.odd or not s.chunks()) for s in SHAPES}
    want = {(m, SKINNY, (b, 16), "", o) for m in (PLAIN, EXPERTS) for b in (16, 32, 64) for o in (False, True)}
    want |= {(m, SKINNY, (16, 64), "", False) for m in (PLAIN, EXPERTS)}
    want |= {(m, DIRECT, (128, 128), "", False) for m in (PLAIN, EXPERTS, GRADIENT)}
    want |= {(m, STAGED, (128, 128), "", True) for m in (PLAIN, EXPERTS, GRADIENT)}
    want |= {(m, STAGED, (128, 128), t, False) for m in (PLAIN, GRADIENT) for t in ("b", "a", "ab")}
    want |= {(PLAIN, TURNED, (256, 128), "b", False), (EXPERTS, STAGED, (128, 128), "b", False)}
    assert want <= have, want - have
    for kernel in (SKINNY, DIRECT, TURNED, STAGED):
        assert any(s.split > 1 for s in SHAPES if s.kernel == kernel)
    for kernel in (DIRECT, STAGED):
        assert any(s.rest for s in SHAPES if s.kernel == kernel)


def test_rest_goes_where_it_pays(plans):
    """Rows past whole tiles leave the launch only where they make a compute unit's share longer and tiles are long."""
    ask = lambda M, N, K: plans([(PLAIN, M, 1, N, K, 1, 1, 0, 1)])[0]  # noqa: E731
    for M, N, K, rest in ((2056, 4096, 4096, 8), (2112, 4096, 4096, 64), (1064, 4096, 4096, 40), (8200, 1024, 2048, 8),
                          (2056, 4096, 1024, 8), (2120, 4096, 4096, 0), (2048, 4096, 4096, 0), (576, 1024, 2048, 0),
                          (264, 4096, 4096, 0), (1088, 1024, 2048, 0), (8256, 4096, 512, 0), (64, 4096, 4096, 0)):
        assert ask(M, N, K)[4] == rest, (M, N, K)


def test_every_plan_holds_together(plans):
    """Over random sizes: kernels get the layouts that they take, slices cover K without an empty one, the rest fits
    the kernel for few rows."""
    rng = random.Random(3)
    size = lambda top: int(2 ** rng.uniform(0, top))  # noqa: E731
    asked = []
    for _ in range(20000):
        mode = rng.choice([PLAIN, PLAIN, EXPERTS, GRADIENT])
        tr = rng.choice([0, 0, 1, 1, 2, 3]) if mode != EXPERTS else rng.choice([0, 1])
        asked.append((mode, size(30), 1 if mode == PLAIN else size(10), size(24), rng.choice([0, size(24), 2 ** 31 - 1]),
                      rng.randint(0, 1), rng.randint(0, 1), tr, int(mode == PLAIN and rng.random() < 0.7)))
    for a, (kernel, bm, bn, split, rest) in zip(asked, plans(asked)):
        mode, rows, n, N, K, direct, small, tr, may = a
        blocks = -(-K // 128)
        assert (kernel == SKINNY) == (rows <= 64 and tr == 0), a
        assert kernel != DIRECT or (direct and small and tr == 0 and bm == bn == 128), a
        assert kernel != TURNED or (direct and small and tr == 1 and mode == PLAIN and (bm, bn) == (256, 128)), a
        assert kernel != STAGED or bm == bn == 128, a
        assert kernel != SKINNY or (bm in (16, 32, 64) and bn == 16 or (bm, bn) == (16, 64) and direct), a
        assert split == 1 or (may and (split - 1) * -(-blocks // split) < blocks), a
        assert rest == 0 or (mode == PLAIN and rest <= 64 and rest == rows % 128 and split == 1 and tr == 0), a
