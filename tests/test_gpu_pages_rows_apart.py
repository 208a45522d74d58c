"""Rows of attention over pages stand apart: a query row of infinities or NaN,
and keys that some rows see and others do not, leave every other row's result as
it is, to the bit, though they share tiles and matrix instructions with it."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from parity_util import TORCH_OF
from quantization_rope_reuse_amd import hkv
from test_gpu_pages import DEV, dev, fresh, ints, say

pytestmark = pytest.mark.gpu
TB, H, GROUP, LEN = 16, 2, 4, 300
SCORES = [dict(), dict(sm_scale=3.0), dict(cap=20.0, sm_scale=0.5), dict(slopes=0.5)]


def made(dtype, n, scores, seed):
    g = np.random.default_rng(seed)
    kp, vp = fresh(g, 20, TB, H, dtype)
    q = dev(g.standard_normal((n, H * GROUP, 128))).to(TORCH_OF[dtype])
    kw = dict(scores, max_queries=n)
    if "slopes" in kw:
        kw["slopes"] = torch.full((H * GROUP,), kw["slopes"], device=DEV)
    return g, q, kp, vp, kw, (ints(np.arange(20)[None]), ints([LEN]), ints([0, n]))


@pytest.mark.parametrize("scores", SCORES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", [2, 7, 70])
def test_infinite_queries(dtype, n, scores):
    say("infinite queries", dtype, n, scores)
    g, q, kp, vp, kw, rest = made(dtype, n, scores, 41)
    clean, cl = hkv.attend_pages(q, kp, vp, *rest, **kw)
    bad = q.clone()
    spoilt = torch.zeros(n, H * GROUP, dtype=torch.bool, device=DEV)
    for i in range(0, n, 3):
        head = int(g.integers(H * GROUP))
        bad[i, head, :: int(g.integers(1, 40))] = [float("inf"), -float("inf"), float("nan")][i // 3 % 3]
        spoilt[i, head] = True
    out, lse = hkv.attend_pages(bad, kp, vp, *rest, **kw)
    assert torch.equal(out[~spoilt], clean[~spoilt]) and torch.equal(lse[~spoilt], cl[~spoilt])


@pytest.mark.parametrize("scores", SCORES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", [7, 70])
def test_infinite_keys(dtype, n, scores):
    """A dim of token 150's key is infinite: rows behind it see it (half of them as
    a score of +infinity, half of -infinity), the others do not."""
    say("infinite keys", dtype, n, scores)
    g, q, kp, vp, kw, rest = made(dtype, n, scores, 42)
    positions = np.sort(np.append(g.integers(100, 150, n // 2), g.integers(150, 200, n - n // 2)))
    kw["positions"] = ints(positions)
    clean, cl = hkv.attend_pages(q, kp, vp, *rest, **kw)
    bad = kp.clone()
    bad[150 // TB, 150 % TB, :, 9] = float("inf")
    out, lse = hkv.attend_pages(q, bad, vp, *rest, **kw)
    fine = dev(positions < 150)
    assert torch.equal(out[fine], clean[fine]) and torch.equal(lse[fine], cl[fine])
    assert not torch.equal(lse[~fine], cl[~fine])
