"""The tiles that rows of attention over pages walk
(csrc/attend_pages_tiles.h, built here for the host): those of the prefix, then
those of what lies behind it, each once, up to the longest cache that the calls
take."""
from __future__ import annotations

import os
import shutil
import subprocess

import numpy as np
import pytest

from conftest import ROOT

SOURCE = r"""
#include <stdio.h>
#include "attend_pages_tiles.h"
int main() {
  int pre, lo, hi, size;
  while (scanf("%d%d%d%d", &pre, &lo, &hi, &size) == 4) {
    const hkv::TileList t = hkv::tiles_of_view(pre, lo, hi, size);
    printf("%d %d %d\n", t.pre, t.lo, t.count);
  }
}
"""
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("needs g++ and the ROCm headers")
    d = tmp_path_factory.mktemp("tiles")
    (d / "tiles.cpp").write_text(SOURCE)
    subprocess.run([gxx, "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    f"-I{ROOT}/quantization_rope_reuse_amd/csrc", str(d / "tiles.cpp"), "-o", str(d / "tiles")],
                   check=True, timeout=120)

    def ask(rows):
        text = "\n".join(" ".join(str(int(x)) for x in r) for r in rows)
        out = subprocess.run([str(d / "tiles")], input=text, capture_output=True, text=True, timeout=60, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return ask


def want(pre, lo, hi, size):
    """(tiles of the prefix, the first one behind it that is walked, how many in all)"""
    p = -(-pre // size)
    first = max(min(lo, hi) // size, p)
    return p, first, p + max(-(-hi // size) - first, 0)


def test_every_tile_once(tiles):
    rows = [(pre, lo, hi, 32) for pre in range(0, 100, 7) for lo in range(0, 170, 13) for hi in range(0, 170, 11)]
    for (pre, lo, hi, size), (p, first, count) in zip(rows, tiles(rows), strict=True):
        walked = [i if i < p else i - p + first for i in range(count)]
        seen = {t // size for t in (*range(pre), *range(min(lo, hi), hi))}
        assert walked == sorted(set(walked)) and seen <= set(walked), (pre, lo, hi)


@pytest.mark.parametrize("size", [32, 64])
def test_longest_caches(tiles, size):
    g = np.random.default_rng(size)
    near = [MOST - i for i in (0, 1, 7, 30, 31, 32, 62, 63, 64, 65, 1000)]
    some = [0, 1, size, *near, *(int(x) for x in g.integers(0, MOST, 6))]
    rows = [(pre, lo, hi, size) for pre in some for lo in some for hi in some]
    for r, (p, first, count) in zip(rows, tiles(rows), strict=True):
        assert (p, first, count) == want(*r), r
        # the last token of any walked tile has 31 bits
        assert count == 0 or (max(p, first + count - p) - 1) * size + size - 1 <= MOST, r
