"""Shapes that between them take every kernel of the block-scaled products in every mode, each
with the kernel that it is there for. tests/test_block_plan.py checks the choice on the CPU,
tests/test_gpu_block_kernels.py the results."""
from __future__ import annotations

SKINNY, DIRECT, TURNED, STAGED = range(4)
PLAIN, EXPERTS, GRADIENT = range(3)


class Shape:
    """kernel: what it is there for; tile: rows and columns of a workgroup; split: slices of K; rest: rows in a
    launch of their own; turn: "a", "b" or "ab", stored with the rows adjacent; odd: rows at odd bytes."""

    def __init__(self, mode, sizes, kernel, tile, split=1, rest=0, turn="", odd=False, b_rows=(1, 128), align=128):
        self.mode, self.sizes, self.kernel, self.tile, self.split, self.rest = mode, sizes, kernel, tile, split, rest
        self.turn, self.odd, self.b_rows, self.align = turn, odd, b_rows, align

    def __repr__(self):
        name = ("plain", "experts", "gradient")[self.mode]
        return "-".join([name, *map(str, self.sizes), ("skinny", "direct", "turned", "staged")[self.kernel],
                         *(["turn_" + self.turn] if self.turn else []), *(["odd"] if self.odd else []),
                         *([f"align{self.align}"] if self.mode == EXPERTS else [])])

    def chunks(self):
        """Whether the operands' rows are 16-byte aligned and hold whole 16-byte chunks."""
        if self.odd:
            return False
        if self.mode == PLAIN:
            M, N, K = self.sizes
        elif self.mode == EXPERTS:
            M, (_, _, _, N, K) = 0, self.sizes
        else:
            _, _, _, M, N = self.sizes
            K = 128
        return (M if "a" in self.turn else K) % 16 == 0 and (N if "b" in self.turn else K) % 16 == 0

    def plan_arguments(self):
        """What the choice is made of (gradients: P from the sizes' capacity)."""
        tr = ("b" in self.turn) + 2 * ("a" in self.turn)
        if self.mode == PLAIN:
            M, N, K = self.sizes
            return PLAIN, M, 1, N, K, int(self.chunks()), 1, tr, 1
        T, k, E, x, y = self.sizes
        n = T * k
        if self.mode == EXPERTS:
            active = max(1, min(E, n))
            return EXPERTS, max(1, n // active), active, x, y, int(self.chunks()), 1, tr, 0
        P = -(-(n + min(E, n) * 127) // 128) * 128
        return GRADIENT, x, E, y, -(-P // E), int(self.chunks()), 1, tr, 0


SHAPES = [
    # few rows: 16, 32 or 64 to a pass, with K in slices, 64 columns to a workgroup, rows at odd bytes
    Shape(PLAIN, (9, 200, 512), SKINNY, (16, 16)),
    Shape(PLAIN, (5, 80, 4096), SKINNY, (16, 16), split=2),
    Shape(PLAIN, (3, 65584, 272), SKINNY, (16, 64)),
    Shape(PLAIN, (30, 100, 272), SKINNY, (32, 16)),
    Shape(PLAIN, (50, 330, 384), SKINNY, (64, 16)),
    Shape(PLAIN, (16, 70, 130), SKINNY, (16, 16), odd=True),
    Shape(PLAIN, (27, 70, 515), SKINNY, (32, 16), odd=True),
    Shape(PLAIN, (64, 70, 2100), SKINNY, (64, 16), odd=True),
    # tiles: few and split, many, a few rows past whole ones
    Shape(PLAIN, (300, 200, 2064), DIRECT, (128, 128), split=4),
    Shape(PLAIN, (2100, 3300, 272), DIRECT, (128, 128)),
    Shape(PLAIN, (2056, 4090, 1040), DIRECT, (128, 128), rest=8),
    Shape(PLAIN, (200, 140, 2083), STAGED, (128, 128), split=4, odd=True),
    Shape(PLAIN, (2100, 3300, 131), STAGED, (128, 128), odd=True),
    Shape(PLAIN, (1064, 4000, 530), STAGED, (128, 128), rest=40, odd=True),
    # stored the other way round
    Shape(PLAIN, (2600, 3280, 400), TURNED, (256, 128), turn="b"),
    Shape(PLAIN, (2000, 3280, 1040), TURNED, (256, 128), split=2, turn="b"),
    Shape(PLAIN, (1500, 608, 272), STAGED, (128, 128), turn="b"),
    Shape(PLAIN, (2100, 3300, 131), STAGED, (128, 128), turn="b"),
    Shape(PLAIN, (304, 200, 1104), STAGED, (128, 128), split=2, turn="a"),
    Shape(PLAIN, (304, 208, 300), STAGED, (128, 128), turn="ab"),
    # experts: a row or a few each, many each, aligned and not
    Shape(EXPERTS, (16, 4, 64, 1032, 272), SKINNY, (16, 64), align=1),
    Shape(EXPERTS, (16, 4, 64, 1032, 272), SKINNY, (16, 64)),
    Shape(EXPERTS, (20, 3, 16, 200, 1552), SKINNY, (16, 16), align=1),
    Shape(EXPERTS, (100, 2, 8, 130, 272), SKINNY, (32, 16), align=1),
    Shape(EXPERTS, (200, 2, 8, 130, 272), SKINNY, (64, 16)),
    Shape(EXPERTS, (30, 2, 8, 130, 133), SKINNY, (16, 16), odd=True),
    Shape(EXPERTS, (100, 2, 8, 130, 133), SKINNY, (32, 16), odd=True),
    Shape(EXPERTS, (200, 2, 8, 130, 133), SKINNY, (64, 16), odd=True, align=1),
    Shape(EXPERTS, (1500, 2, 8, 1100, 272), DIRECT, (128, 128), align=1),
    Shape(EXPERTS, (1500, 2, 8, 1100, 272), DIRECT, (128, 128)),
    Shape(EXPERTS, (500, 2, 4, 300, 1552), DIRECT, (128, 128)),
    Shape(EXPERTS, (500, 2, 4, 300, 133), STAGED, (128, 128), odd=True, align=1),
    Shape(EXPERTS, (500, 2, 4, 304, 272), STAGED, (128, 128), turn="b"),
    # gradients: few rows of C, many; more than 1024 of k; every layout
    Shape(GRADIENT, (300, 2, 4, 48, 200), SKINNY, (64, 16)),
    Shape(GRADIENT, (300, 2, 4, 12, 200), SKINNY, (16, 16)),
    Shape(GRADIENT, (300, 2, 4, 30, 200), SKINNY, (32, 16), odd=True),
    Shape(GRADIENT, (300, 2, 4, 300, 600), DIRECT, (128, 128)),
    Shape(GRADIENT, (2000, 2, 3, 200, 300), DIRECT, (128, 128)),
    Shape(GRADIENT, (300, 2, 4, 140, 200), STAGED, (128, 128), odd=True),
    Shape(GRADIENT, (300, 2, 4, 300, 208), STAGED, (128, 128), turn="b"),
    Shape(GRADIENT, (2000, 2, 3, 208, 304), STAGED, (128, 128), turn="a"),
    Shape(GRADIENT, (300, 2, 4, 208, 304), STAGED, (128, 128), turn="ab"),
]
