"""Attention over records along every way the rows kernel shares out its work
(attend_paths.py; test_attend_share.py holds that they are reached), with the
tolerances of test_gpu_serve.py (check_attend)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from attend_paths import blocks_of, cases, name_of
from parity_util import TORCH_OF
from quantization_rope_reuse_amd import hkv
from test_gpu_serve import DEV, check_attend, pool, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", cases(), ids=name_of)
def test_path(case):
    say("path", name_of(case))
    _, fmt, dtype, tb, h, group, lens, asks, moved, _ = case
    g = np.random.default_rng([tb, h, group, moved])
    held = [-(-n // tb) for n in lens]
    table = np.full((len(lens), blocks_of(lens, tb)), -1, np.int32)
    ids, at = g.permutation(sum(held) + 2).astype(np.int32), 0
    for r, n in enumerate(held):
        table[r, :n] = ids[at:at + n]
        at += n
    rec = pool(g, fmt, sum(held) + 2, tb, h)
    table[0, 1] = -1                     # a block left out
    q = torch.from_numpy(1.5 * g.standard_normal((sum(asks), h * group, 128))).to(DEV, TORCH_OF[dtype])
    kw = {}
    if moved:
        dm = g.integers(-3000, 3001, table.shape).astype(np.int32)
        dm[:, 3:7] = dm[:, 3:4]
        kw = dict(delta_m=dm, rope_base=1e4, pairs="interleaved" if tb == 16 else "half_split")
    check_attend(q, rec, fmt, tb, h, table, lens, np.concatenate([[0], np.cumsum(asks)]), name_of(case),
                 max_queries=max(asks), **kw)


@pytest.mark.parametrize("fmt", ["int4", "fp8"])
@pytest.mark.parametrize("tb", [64, 16, 7])
def test_records_beyond_32_bits(fmt, tb):
    """Records 600 MB apart, the last from byte 4.8e9 on; few rows, a pair of
    heads, a prompt's rows."""
    say("far records", fmt, tb)
    g = np.random.default_rng(tb)
    h, nb, stride = 2, 9, 600 * 1024 * 1024
    rb = hkv.record_bytes(fmt, tb, h)
    rec = torch.empty((nb - 1) * stride + rb, dtype=torch.uint8, device=DEV).as_strided((nb, rb), (stride, 1))
    x = torch.from_numpy(g.standard_normal((2, nb * tb, h, 128)).astype(np.float32)).to(DEV)
    hkv.append_tokens(x[0], x[1], torch.arange(nb * tb, device=DEV), rec, fmt, tb)
    for n, group, room in ((1, 4, nb), (2, 4, 20000 // tb), (35, 64, nb)):
        table = np.full((1, room), -1, np.int32)
        table[0, :nb] = np.arange(nb - 1, -1, -1)
        q = torch.from_numpy(1.5 * g.standard_normal((n, h * group, 128))).to(DEV, torch.bfloat16)
        for dm in (None, np.full(table.shape, 50, np.int32)):
            check_attend(q, rec, fmt, tb, h, table, [nb * tb - 3], [0, n], f"{n} queries", max_queries=n, delta_m=dm)
