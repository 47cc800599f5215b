"""Which tile shape the expert product takes for a call, and how many tiles a persistent workgroup
takes one after the other: the host's rule of moe_experts.hip in Python, with its table of costs read
from the source, so that a test can tell whether its cases still reach what they are there for."""
import os
import re

from conftest import ROOT

SOURCE = os.path.join(ROOT, "combine_moe_route_03_amd", "csrc", "moe_experts.hip")
KSTEP, XCDS, CUS = 128, 8, 256


def table():
    """(rows, channels, slots, step, alone, tile) of each shape, and the limit for few tiles."""
    text = open(SOURCE).read()
    body = re.search(r"kTiles\[\] = \{(.*?)\n\};", text, re.S).group(1)
    rows = [tuple(float(v.rstrip("f")) for v in r.split(",")) for r in re.findall(r"\{(.*?)\}", body)]
    few = int(re.search(r"kFewTiles = (\d+);", text).group(1))
    return [(int(m), int(n), int(s), *t) for m, n, s, *t in rows], few


def up(a, b):
    return -(-a // b)


def shape(R, E, N, K, act):
    """(rows, channels) of the tiles that R rows of E experts take, or None: the kernel of few rows."""
    tiles, few = table()
    n_w, experts = (2 * N if act == "swiglu" else N), min(E, R)
    if (R // 32 + experts) * up(n_w, 128) < few:
        return None
    best = None
    for bm, bn, slots, step, alone, tile in tiles:
        n = max(R // bm + experts // 2, experts) * up(n_w, bn)
        time = up(n, slots) * (up(K, KSTEP) * (alone if n <= 256 else step) + tile)
        if best is None or time < best[0]:
            best = time, bm, bn
    return best[1:]


def most_of_workgroup(bm, bn, counts, N, act):
    """Tiles of the workgroup that takes the most, for shapes with persistent workgroups."""
    blocks = up(N, bn // 2 if act == "swiglu" else bn)
    R, E = int(sum(counts)), len(counts)
    most = (R // bm + min(E, R)) * blocks
    workgroups = CUS * (2 if (bm, bn) == (128, 128) else 1)
    workgroups = min(up(most, XCDS) * XCDS, workgroups)
    return up(up(sum(up(int(c), bm) for c in counts) * blocks, XCDS), workgroups // XCDS)


# (rows, channels of the tile), T, E, N, K, kind, act: workgroups that take 2 to 4 tiles, with rows of
# out on and off 16 bytes, whole and ragged K of two steps and more
SEVERAL = [
    ((64, 256), 13214, 100, 144, 224, "even", "none"),
    ((64, 256), 1045, 4, 1616, 144, "even", "swiglu"),
    ((64, 256), 13214, 100, 401, 256, "uneven", "none"),
    ((128, 128), 13265, 200, 296, 176, "even", "none"),
    ((128, 128), 17168, 100, 264, 144, "uneven", "swiglu"),
    ((128, 256), 9000, 4, 2056, 1424, "uneven", "none"),
    ((128, 256), 9000, 4, 1032, 1424, "uneven", "swiglu"),
    ((128, 256), 4264, 16, 1456, 784, "even", "none"),
    ((128, 256), 2171, 16, 2515, 832, "even", "none"),
    ((128, 256), 8332, 32, 267, 912, "even", "swiglu"),
    ((256, 256), 1098, 4, 8232, 288, "even", "none"),
    ((256, 256), 4000, 1, 2056, 272, "even", "swiglu"),
]

# more tiles than the ring that hands them from the loads to the products has places
MANY = [
    ((64, 256), 9251, 384, 728, 144, "even", "swiglu", True),
    ((64, 256), 5798, 200, 3512, 16, "even", "none", False),
    ((128, 128), 17119, 384, 1400, 160, "even", "none", True),
    ((128, 256), 15212, 100, 1416, 1344, "even", "swiglu", True),
    ((256, 256), 13212, 4, 5928, 400, "even", "swiglu", False),
]
RING = 8
