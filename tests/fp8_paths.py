"""Shapes that take the FP8 product down each of its ways, and which way a shape takes on a
GB300 (152 SMs)."""
import nvfp4_frozen_projection_gb300 as pk

SHAPES = [
    # few tokens: 8 or 16 of them a CTA, 16, 8 or 4 warps
    (2, 1040, 2064), (1, 4096, 2064), (8, 4112, 1040), (5, 2560, 4112), (3, 8208, 1040),
    (11, 1040, 1040), (40, 1040, 2064), (70, 2064, 528),
    # a CTA a tile: boxes of X lower than the tile, outputs narrower than the tile
    (24, 16384, 2048), (8, 16384, 16384), (127, 12304, 1040), (300, 4240, 2064),
    (1500, 112, 528), (1100, 16, 16),
    # clusters of two, three and four a tile
    (60, 8192, 4112), (500, 2048, 4112), (120, 4880, 2064), (300, 1600, 4112), (100, 4096, 2192),
    (333, 1040, 2064), (1100, 64, 8192),
    # pairs: with a last tile whose second CTA, or second 128 columns, lie past the output
    (2100, 4080, 1040), (2304, 4080, 1040), (4296, 2688, 2064), (4100, 2688, 2064),
    # a last wave of halves: the second half past the output, and not
    (4700, 2176, 6160), (4800, 2176, 6160), (4700, 2304, 6160), (4800, 2304, 6160),
]


def instance(m, n, k):
    """The way, and what of the shape makes a difference on it."""
    way, share, whole = pk.pact_test_fp8_plan(m, n, k)
    if way == "few":
        return way, 8 if m <= 8 else 16, share
    if way == "tiles":
        return way, m < 128, n < 128
    if way == "shared":
        return way, share, m < 128
    return "halves" if whole else way, 0 < m % 256 <= 128, 0 < n % 256 <= 128


ALL = ({("few", t, w) for t in (8, 16) for w in (4, 8, 16)}
       | {("tiles", True, False), ("tiles", False, False), ("tiles", False, True)}
       | {("shared", s, low) for s in (2, 3, 4) for low in (True, False)}
       | {(w, m, n) for w in ("pairs", "halves") for m in (True, False) for n in (True, False)})
