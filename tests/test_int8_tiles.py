"""The choice of tiles of the 8-bit integer products, read from the kernel's source: the GPU tests' sizes reach every
tile with every number of row blocks that its last tile may have, and no size asks for a launch of 2^32 threads."""
from __future__ import annotations

import os
import re

from tests.test_gpu_int8_tiles import TILES
from weight_only_quantization_quantize_amd import build as woq_build

SOURCE = open(os.path.join(woq_build.CSRC, "int8_gemm.hip")).read()
UNITS = 256


def models():
    """(BM, BN, fixed, tile, stage, threads, rows of a wave row of blocks) of each tile, in the order of their numbers."""
    table = re.search(r"kModels\[\] = \{(.*?)\};", SOURCE, re.S).group(1)
    rows = [tuple(map(float, m)) for m in re.findall(r"\{" + ", ".join([r"([\d.]+)"] * 5) + r"\}", table)]
    tiles = re.findall(r"(?:case (\d+)|default): return run\(Int8Tile<([^>]*)>", SOURCE)
    assert len(rows) == len(tiles) and [int(n or len(rows) - 1) for n, _ in tiles] == list(range(len(rows)))
    out = []
    for (bm, bn, *time), (_, args) in zip(rows, tiles):
        tm, tn, wn, _, kg, _, _, wm = [*map(int, args.split(",")), 2, 2][:8]
        assert (bm, bn) == (32 * wm * tm, 32 * wn * tn)
        out.append((int(bm), int(bn), *time, 64 * wm * wn * kg, 32 * wm))
    return out


MODELS = models()


def choose(M, N, K):
    def time(m):
        rounds = (-(-M // m[0]) * -(-N // m[1]) + UNITS - 1) // UNITS
        return m[2] + rounds * (m[3] + m[4] * -(-K // 128))
    return min(range(len(MODELS)), key=lambda i: time(MODELS[i]))


def test_sizes_reach_every_tile_and_every_last_one():
    wanted = {(i, b) for i, m in enumerate(MODELS) for b in range(1, m[0] // m[6] + 1)}
    for part in (TILES, [s for s in TILES if s[2] > 5 * 128]):  # of one stage and of more than there are in LDS
        reached = set()
        for M, N, K in part:
            assert M > 4 and M % 16 and N % 16
            i = choose(M, N, K)
            reached.add((i, -(-(M % MODELS[i][0]) // MODELS[i][6])))
        assert reached == wanted


def test_launches_stay_below_32_bits_of_threads():
    """Outputs of up to 2^25 blocks of 64 x 64 are taken (include/woq.h's limits of M and N beside)."""
    sizes = sorted({(1 << i) + d for i in range(3, 29) for d in (-1, 0, 1)} | {3 * (1 << i) for i in range(2, 27)})
    for M in (s for s in sizes if 5 <= s <= 1 << 28):
        for N in (s for s in sizes if s <= 1 << 28):
            if -(-M // 64) * -(-N // 64) > 1 << 25:
                continue
            for K in (16, 128, 1024, 16384):
                m = MODELS[choose(M, N, K)]
                assert (-(-M // m[0]) * -(-N // m[1]) + 7) * m[5] < 1 << 32, (M, N, K)
