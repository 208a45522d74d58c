"""How the work of attention over pages is shared out
(csrc/attend_pages_share.h, host code built here): the calls of
attend_pages_paths.py reach the paths they name, so that a moved threshold does
not take a path's tests away unseen; launches and workspaces stay within what
the kernels take."""
from __future__ import annotations

import os
import shutil
import subprocess

import numpy as np
import pytest

from attend_pages_paths import CASES, blocks_of
from conftest import ROOT

SOURCE = r"""
#include <stdio.h>
#include "attend_pages_share.h"
int main() {
  int tb, h, r, mb, mq, n, hq, slanted;
  while (scanf("%d%d%d%d%d%d%d%d", &tb, &h, &r, &mb, &mq, &n, &hq, &slanted) == 8) {
    hkv_requests q = {};
    q.n_requests = r; q.max_blocks = mb; q.max_queries = mq;
    const hkv::PageShare s = hkv::page_share_of(hkv::Geometry{1, 64, tb, h, tb * h}, q, n, hq, slanted != 0);
    printf("%d %d %d %d %lld %lld %lld %d\n", s.splits, s.ranges, s.min_tiles, s.part_rows, (long long)s.rows,
           (long long)s.items, (long long)hkv::page_share_bytes(s), hkv::page_join_sets(s, r));
  }
}
"""
FIELDS = ("splits", "ranges", "min_tiles", "part_rows", "rows", "items", "bytes", "sets")


@pytest.fixture(scope="module")
def shares(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("needs g++ and the ROCm headers")
    d = tmp_path_factory.mktemp("share")
    (d / "share.cpp").write_text(SOURCE)
    subprocess.run([gxx, "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", f"-I{ROOT}/include",
                    f"-I{ROOT}/quantization_rope_reuse_amd/csrc", str(d / "share.cpp"), "-o", str(d / "share")],
                   check=True, timeout=120)

    def ask(rows):
        text = "\n".join(" ".join(str(int(x)) for x in r) for r in rows)
        out = subprocess.run([str(d / "share")], input=text, capture_output=True, text=True, timeout=60, check=True).stdout
        return [dict(zip(FIELDS, map(int, line.split()))) for line in out.splitlines()]
    return ask


def test_cases_reach_their_paths(shares):
    rows = [(tb, h, len(lens), blocks_of(lens, tb), max(asks), sum(asks), h * group, positions)
            for _, tb, h, group, lens, asks, positions, _ in CASES]
    got = [("chunk", s["splits"]) if s["splits"] else ("rows", s["ranges"], s["sets"]) for s in shares(rows)]
    for c, share in zip(CASES, got, strict=True):
        assert share == c[-1], c


def test_sizes_stay_in_range(shares):
    g = np.random.default_rng(5)
    rows = []
    for _ in range(3000):
        h = int(2 ** g.uniform(0, 12))
        group = int(2 ** g.uniform(0, 7))
        r = int(2 ** g.uniform(0, 16)) - 1
        n = int(min(2 ** g.uniform(0, 20), (2 ** 31 - 1) // (h * group)))
        tb = int(2 ** g.uniform(0, 8))
        mb = int(min(2 ** g.uniform(0, 24), (2 ** 31 - 1) // tb))
        rows.append((tb, h, max(r, 1), mb, int(2 ** g.uniform(0, 20)), n, h * group, g.integers(2)))
    for x, s in zip(rows, shares(rows), strict=True):
        tb, h, r, mb, mq, n, hq, _ = x
        assert s["items"] >= 0 and s["rows"] >= 0 and 1 <= s["sets"] <= 16, x
        assert s["splits"] * h <= 65535 and s["ranges"] * h <= max(256, h), x
        if s["splits"] > 1:
            assert s["rows"] == s["splits"] * n * hq and s["bytes"] >= 516 * s["rows"] + 4 * n * hq, x
        if s["ranges"]:
            # the dealing's sums have 32 bits; the join has 16 lanes for each row a request might have
            assert r <= 1024 and r * s["items"] * -(-mb * tb // 32) < 2 ** 30 and min(mq, n) * hq <= 2 ** 20, x
            assert s["bytes"] >= 516 * s["rows"] + 4 * (r + 2) and s["part_rows"] <= 32, x
        if not s["rows"]:
            assert s["bytes"] == 0, x
