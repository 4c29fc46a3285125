"""Sizes that together take every tensor-core kernel of the centre network's linear layer and its
gradients, and the name of the kernels that a size takes (from the library's own plan; no GPU)."""

import ctypes

from virtual_noise_perturbed_gb300 import _lib

# (type, gradients?) -> (rows, in, out), aligned, each for a kernel that none of the others takes.
SIZES = {
    ("fp32", False): [
        (32, 18264, 32), (32, 17474, 31), (280, 16480, 32), (408, 18281, 35), (2344, 4440, 32), (1113, 8382, 30),
        (10, 9, 63281),
        (64, 64, 64), (64, 79, 65), (64, 36970, 64), (68, 75, 11004), (72, 64, 31168), (91, 64, 33027),
        (147, 44719, 211), (168, 66, 11074), (192, 64, 11162), (270, 4957, 704), (300, 257, 130), (344, 69, 10347),
        (520, 130, 2056), (1000, 72, 4104), (2880, 64, 64), (12566, 64, 64), (18816, 64, 192), (19015, 87, 142),
        (29568, 69, 78),
    ],
    ("fp32", True): [
        (37312, 40, 32), (5232, 32, 1032), (2464, 56, 4649),
        (1, 23090, 1), (64, 64, 64), (64, 65, 22454), (64, 79, 65), (64, 100, 19776), (64, 131, 3368),
        (64, 600, 6010), (64, 47299, 70), (70, 1231, 421), (72, 4095, 512), (72, 4095, 1031), (72, 7040, 64),
        (76, 416, 2734), (152, 64, 9173), (960, 2120, 65), (2056, 130, 640), (2240, 576, 74), (3136, 361, 64),
        (3706, 1048, 64), (4608, 278, 88), (17700, 137, 64), (29568, 69, 78), (47859, 64, 75),
    ],
    ("bf16", False): [
        (64, 64, 64), (64, 79, 65), (64, 560, 64), (64, 3712, 64), (72, 64, 25712), (72, 520, 100), (72, 1000, 72),
        (128, 448, 10176), (640, 257, 130), (640, 3000, 72), (645, 13343, 152), (742, 436, 2609), (1767, 64, 280),
        (3301, 64, 653), (18816, 64, 192), (19015, 87, 142), (23261, 184, 84),
    ],
    ("bf16", True): [
        (64, 64, 64), (64, 79, 65), (64, 1040, 3408), (72, 130, 3000), (72, 7040, 64), (74, 20224, 64),
        (79, 142, 17335), (80, 21206, 73), (82, 1208, 13444), (128, 64, 2751), (192, 72, 26240), (384, 65, 7168),
        (400, 9903, 128), (448, 10680, 119), (3000, 72, 100), (3112, 144, 68), (3706, 1048, 64), (4608, 312, 431),
        (9096, 139, 481), (16390, 130, 640), (17700, 137, 64), (22080, 64, 192),
    ],
}

# (rows, in, out) whose weight gradients in bf16 take pairs' tiles of 32, 48, .. 256 columns.
WIDTHS = [
    (1100, 640, n) for n in (520, 808, 1208, 1608, 2008, 2408, 2808, 3208, 3608, 4008)] + [
    (1100, 1024, n) for n in (3352, 3656, 3960)] + [(1100, 2048, n) for n in (2024, 2168)]


def plan(rows, n_in, n_out, kind, backward, aligned=True, act=0):
    p = (ctypes.c_int32 * 10)()
    dt = _lib.VN_BF16 if kind == "bf16" else _lib.VN_F32
    assert _lib.load().vn_testhook_linear_plan(rows, n_in, n_out, dt, act, aligned, backward, p) == 0
    return list(p)


def kernels(rows, n_in, n_out, kind, backward, aligned=True, act=0):
    """The kernels of a call. A pair of CTAs stores its rows by TMA ("staged") or not, has one tile or
    several, and its halves of a tile end on a 64-wide block or within one."""
    p = plan(rows, n_in, n_out, kind, backward, aligned, act)
    per = 8 if kind == "bf16" else 4
    if p[0] == 0:
        return {(kind, "rows", aligned and n_in % per == 0)}
    if p[0] == 2:
        # fp32 sums over a long share of k are taken in pieces.
        shares = [-(-n // 64 >> l) for n, l in ((n_out if backward else n_in, p[2]), (rows if backward else 0, p[3]))]
        long = kind == "fp32" and max(shares) > (16 if p[1] == 128 else 32)
        packs = aligned and n_in % per == 0 and (not backward or n_out % per == 0)
        return {(kind, "gather", "gradients" if backward else "forward", p[1], "packs" if packs else "any", "pieces" if long else "whole")}
    found = set()
    products = [("dx", p[4:7], n_in, rows), ("dw", p[7:10], n_in, n_out)] if backward else [("y", p[4:7], n_out, rows)]
    for name, (pair, columns, split), np, nq in products:
        if pair:
            many = -(-np // 256) * -(-nq // columns) > 76
            found.add((kind, "pair", name, "staged" if np % per == 0 else "unstaged", "many" if many else "one",
                       "blocks" if columns % 128 == 0 else "parts"))
        else:
            found.add((kind, "single", name, columns, "split" if split else "whole"))
    return found
