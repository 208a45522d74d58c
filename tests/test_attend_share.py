"""How attention's work is shared out (csrc/attend_share.h, host code built
here): the calls of attend_paths.py reach the paths they name, so that a moved
threshold does not take a path's tests away unseen; sizes of workspaces and
launches stay within what the kernels take."""
from __future__ import annotations

import os
import shutil
import subprocess

import numpy as np
import pytest

from attend_paths import PROMPTS, blocks_of, cases
from conftest import ROOT

FMT = {"fp8": 0, "int4": 1}
DT = {"f32": 0, "f16": 1, "bf16": 2}
SOURCE = r"""
#include <stdio.h>
#include "attend_share.h"
int main() {
  int fmt, moved, nb, tb, h, r, mb, mq, n, hq, dt;
  while (scanf("%d%d%d%d%d%d%d%d%d%d%d", &fmt, &moved, &nb, &tb, &h, &r, &mb, &mq, &n, &hq, &dt) == 11) {
    hkv_requests q = {};
    q.n_requests = r; q.max_blocks = mb; q.max_queries = mq;
    const hkv::Share s = hkv::share_of(fmt, moved != 0, hkv::Geometry{1, nb, tb, h, tb * h}, q, n, hq, dt);
    printf("%d %d %d %d %d %d %d %d %lld %lld %lld\n", s.splits, s.hp, s.nt, s.set_heads, s.head_sets, s.ranges,
           s.min_tiles, s.part_rows, (long long)s.rows, (long long)s.items, (long long)hkv::share_bytes(s, q));
  }
}
"""
FIELDS = ("splits", "hp", "nt", "set_heads", "head_sets", "ranges", "min_tiles", "part_rows", "rows", "items", "bytes")


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
    rows = [(FMT[fmt], moved, 64, tb, h, len(lens), blocks_of(lens, tb), max(asks), sum(asks), h * group, DT[dtype])
            for _, fmt, dtype, tb, h, group, lens, asks, moved, _ in cases()]
    for c, s in zip(cases(), shares(rows), strict=True):
        got = (s["hp"], s["nt"], s["set_heads"], s["ranges"] > 0)
        assert s["splits"] == 0 and got == c[9], c

    rows = [(FMT[fmt], moved, 64, tb, h, len(lens), blocks_of(lens, tb), max(asks), sum(asks), h * group, DT[dtype])
            for fmt, dtype, tb, h, group, lens, asks, _ in PROMPTS for moved in (False, True)]
    for c, s in zip([c for c in PROMPTS for _ in range(2)], shares(rows), strict=True):
        assert s["splits"] > 0 and (s["splits"] > 1) == c[7], (c, s["splits"])
    # the paired heads of test_gpu_nonfinite.py
    for s in shares([(fmt, moved, 4, tb, 8, 1, -(-4200 // tb), 2, 2, 32, dt) for fmt in (0, 1) for moved in (0, 1)
                     for tb in (64, 16, 7) for dt in (0, 1, 2)]):
        assert s["splits"] == 0 and s["hp"] == 2


def test_sizes_hold(shares):
    """Over calls of all sizes: heads divide, a range's partial rows and the
    launch fit, and the prompt kernel's grid too."""
    g = np.random.default_rng(0)
    rows = []
    for _ in range(4000):
        h, r = int(g.choice([1, 2, 3, 5, 8, 16, 64, 4096])), int(np.exp(g.uniform(0, np.log(65535))))
        group = int(g.choice([1, 2, 4, 5, 8, 16, 64]))
        tb = int(g.choice([1, 7, 16, 32, 64, 1024]))
        mb = int(min(np.exp(g.uniform(0, np.log(2 ** 31 - 1))), (2 ** 31 - 1) // tb))
        n = int(min(np.exp(g.uniform(0, np.log(10 ** 6))) + 1, (2 ** 31 - 1) // (h * group)))
        rows.append((g.integers(2), g.integers(2), 64, tb, h, r, mb, int(g.choice([1, 5, n, 2 ** 31 - 1])), n, h * group,
                     g.integers(3)))
    for (fmt, moved, _, tb, h, r, mb, mq, n, hq, dt), s in zip(rows, shares(rows), strict=True):
        queries = min(mq, n)
        group_rows = queries * (hq // h)
        assert s["items"] >= 1 and s["bytes"] >= 0
        if s["splits"]:
            assert group_rows > 384 and s["items"] * 256 >= group_rows and h * s["splits"] <= 65535
            assert s["rows"] == (s["splits"] * n * hq if s["splits"] > 1 else 0)
            assert s["splits"] <= 256
        else:
            assert group_rows <= 384 or (n * (hq // h) < 256 * r and queries * hq * r <= 1 << 19)
            heads = s["set_heads"] * s["hp"]
            assert heads * s["head_sets"] == h and heads in (1, 2)
            item = 16 * s["nt"] // s["hp"]
            assert s["items"] * item >= group_rows and s["part_rows"] == min(item, group_rows)
            assert s["rows"] == s["ranges"] * 2 * h * s["part_rows"]
            if s["ranges"]:
                assert r <= 1024 and s["ranges"] <= 512 and queries * hq <= 1 << 20
                tiles = max(1, -(-mb * tb // 32))
                assert r * s["items"] * tiles < 1 << 30
