"""The grid of a tree attention never has more CTAs than the workspace has parts for, whatever a launcher asks for. No GPU needed."""
import glob
import os
import subprocess

import numpy as np
import pytest

from kv_cache_compression_gb300 import build as kbuild
from kv_cache_compression_gb300 import draft as kd

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    kbuild.build()
    objects = sorted(glob.glob(os.path.join(kbuild._BUILD, "*.o")))
    exe = str(tmp_path_factory.mktemp("grid") / "tree_grid")
    subprocess.run([kbuild.nvcc(), *kbuild.ARCH, *kbuild.FLAGS, os.path.join(HERE, "tree_grid.cu"), *objects, "-o", exe], check=True)

    def run(calls):
        text = "".join(" ".join(map(str, c)) + "\n" for c in calls)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split()
        return list(zip(map(int, out[::2]), map(int, out[1::2])))
    return run


def shapes(n):
    rng = np.random.default_rng(3)
    def size(hi):
        return int(np.exp(rng.uniform(0, np.log(hi + 1))))
    found = [(65535, 1, 1, 64, 1, 300), (1, 1, 1, 128, 1 << 22, 17), (1, 16, 16, 128, 1, 257), (1, 17, 1, 64, 1, 1)]
    while len(found) < n:
        B, H, G, T, cap = size(300), size(64), size(8), size(2000), size(1 << 20)
        if B * H <= 65535 and B * H * G * T <= 1 << 22:
            found.append((B, H * G, H, int(rng.choice([64, 128])), T, cap))
    return found


def test_parts_end_inside_the_workspace(cut):
    """Each kernel's passes and tiles, for its own grid and for larger ones."""
    calls = []
    for B, Hq, H, d, T, cap in shapes(1500):
        rows = Hq // H * T
        # fp32 instructions; mma.sync (up to sixteen rows, over 8 bits 32); tcgen05 (more)
        kinds = [(8 if rows <= 8 else 32, 64, 64, 304)]
        if rows <= 32:
            kinds += [(8 if rows <= 8 else 16, 16, 16, 304), (8 if rows <= 8 else 16, 32, 16, 304)]
        if rows > 16:
            kinds += [(q, 128, 128, 152) for q in (128, 256) if rows > q // 2 or q == 128]
        for tile_q, tile, fresh, ctas in kinds:
            passes = -(-rows // tile_q)
            for siblings in {1, passes} if 4 * passes <= ctas else {1}:
                for asked in (ctas, 320, 608, 1 << 20):
                    calls.append((B, Hq, H, d, T, cap, tile_q, siblings, tile, fresh, asked - asked % siblings))
    for call, (ctas, end) in zip(calls, cut(calls)):
        B, Hq, H, d, T, cap, tile_q, siblings, tile, fresh, asked = call
        room = kd.tree_workspace_size(B, Hq, H, d, T, cap)
        assert end <= room, call
        assert ctas >= 1 and (room == 0 or (ctas <= 320 and ctas % siblings == 0)), call
        if room and asked <= (152 if tile_q >= 128 else 304):   # a kernel's own grid is not cut down
            passes = -(-(Hq // H * T) // tile_q)
            tiles = B * H * passes * (-(-cap // tile) + -(-T // fresh))
            assert ctas == min(asked, tiles - tiles % siblings), call
