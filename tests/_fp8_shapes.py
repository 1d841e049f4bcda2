"""A shape (M, N, K) for every kernel of the FP8 product, with ends of rows, columns and K
inside a tile, and for the tile kernels one whose K passes 64 stages of 128. The names are
those of csrc/fp8_plan.hpp; test_fp8_plan.py holds the table to the plan."""

# kernel of 16-bit outputs, K splits, columns split off
SHAPES = {
    "kRows8": (5, 199, 656), "kRows8Deep": (5, 4101, 2064), "kRows8Narrow": (6, 199, 2064),
    "kRows16": (12, 199, 656), "kRows16Deep": (12, 4101, 2064), "kRows16Narrow": (13, 199, 2064),
    "kRows32": (20, 199, 656), "kRows32Deep": (20, 4101, 2064), "kRows32Narrow": (21, 199, 2064),
    "kTile64": (40, 259, 656), "kTile64 split": (40, 259, 2064), "kTile64x128": (60, 16387, 656),
    "kTile64x192": (60, 34003, 656), "kTile128": (1500, 4999, 656), "kTile128Deep": (300, 9001, 656),
    "kTile128Deep split": (201, 3839, 8208), "kTile128x192": (130, 20001, 656), "kTile256x192": (300, 23990, 272),
    "kTile256": (2000, 8190, 272), "kTile256 tail": (1990, 8450, 272),
}
LONG = {
    "kTile64 split": (64, 5120, 17408), "kTile64x128": (60, 24500, 17424), "kTile64x192": (60, 34003, 8464),
    "kTile128": (2000, 4095, 17424), "kTile128Deep": (700, 4097, 17424), "kTile128x192": (1000, 5119, 17424),
    "kTile256x192": (2047, 5120, 17408), "kTile256": (2000, 8190, 17424), "kTile256 tail": (1990, 8450, 8464),
}
