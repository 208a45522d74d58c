"""Attention over records whose scores are so large that fp32 holds no
fraction of them: results stay finite, and where one token leads by more than
the scores' own error (160 * 2^-24 of the largest sum of |q k|, as in
test_gpu_serve.py) plus 100, the result is that token's value: off by the
weight's rounding, 2^-11 for bf16 results and 2^-22 for the others, by 2^-20
for exp2 and the sum, and by the result's rounding.  Elsewhere no result is
larger than the largest value seen."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
from parity_util import TORCH_OF, host_f64
from quantization_rope_reuse_amd import hkv
from test_gpu_serve import DEV, HALF, TINY, dev, on_device, say

pytestmark = pytest.mark.gpu


def records(g, fmt, nb, tb, h):
    """Values of tokens from 2^-10 to 2^10 in size, some tokens zero."""
    x = g.standard_normal((2, nb, tb, h, 128))
    x[1] *= np.exp2(g.integers(-10, 11, (nb, tb, h, 1)))
    x[1, :, 5 % tb] = 0
    x[1, 0] = 0
    rec = O.put(x[0][None], x[1][None], np.arange(nb), fmt)[0]
    kd, vd = (a[0].astype(np.float64) for a in O.dequant_records(rec, fmt, tb, h))
    return on_device(rec[0], fmt, tb, h), kd, vd


# queries, key heads, query heads per key head, block_tokens, blocks: one and
# two tiles of 16 rows, a pair of heads, more tokens than one workgroup takes,
# a prompt, one whose tokens are cut
SHAPES = [(1, 1, 4, 16, 8), (7, 2, 4, 32, 6), (1, 8, 4, 64, 200), (3, 8, 8, 64, 200), (2, 2, 8, 16, 90), (110, 1, 4, 16, 8),
          (200, 1, 2, 64, 21), (37, 1, 128, 16, 8), (37, 1, 128, 64, 21)]


@pytest.mark.parametrize("fmt,dtype", [("int4", "bf16"), ("int4", "f16"), ("fp8", "f32"), ("fp8", "bf16")])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_far_scores(fmt, dtype, shape):
    say("far scores", fmt, dtype, shape)
    n, h, group, tb, nb = shape
    g = np.random.default_rng(list(shape))
    rec, kd, vd = records(g, fmt, nb, tb, h)
    table = g.permutation(nb).astype(np.int32)
    length = nb * tb - 3
    k = kd[table].reshape(-1, h, 128)[:length]
    v = vd[table].reshape(-1, h, 128)[:length]
    q = torch.from_numpy(np.clip(g.standard_normal((n, h * group, 128)), -2, 2)).to(DEV, TORCH_OF[dtype])
    x = host_f64(q).reshape(n, h, group, 128)
    raw = np.einsum("nhgd,thd->nhgt", x, k)
    reach = np.einsum("nhgd,thd->nhgt", np.abs(x), np.abs(k)).max(-1)
    w = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -22
    for power in range(15, 42, 2):
        scale = 2.0 ** power
        got, lse = hkv.attend_records(q, rec, fmt, tb, h, dev(table[None]), dev(np.array([length], np.int32)),
                                      dev(np.array([0, n], np.int32)), max_queries=n, causal=False, sm_scale=scale)
        torch.cuda.synchronize()
        got, lse = host_f64(got).reshape(n, h, group, 128), host_f64(lse).reshape(n, h, group)
        what = f"scale 2^{power}"
        assert np.isfinite(got).all() and np.isfinite(lse).all(), \
            f"{what}: {(~np.isfinite(got)).any(-1).sum()} rows of {lse.size} not finite"
        ds = reach * scale * 160 * 2.0 ** -24
        s = raw * scale
        top = s.max(-1)
        assert (np.abs(lse - top) <= ds + np.log(length) + 2.0 ** -20 + 2.0 ** -22 * np.abs(top)).all(), f"{what}: lse"
        eps = w + 2.0 ** -20 + HALF[dtype]
        most = np.abs(v).max(0)[None, :, None]
        assert (np.abs(got) <= most * (1 + eps) + TINY[dtype]).all(), f"{what}: larger than any value"
        alone = (s < (top - 2 * ds - 100)[..., None]).sum(-1) == length - 1
        assert alone.mean() > 0.5
        want = np.moveaxis(v, 0, 1)[np.arange(h)[None, :, None], s.argmax(-1)]
        ok = np.abs(got - want) <= np.abs(want) * eps + TINY[dtype]
        assert ok[alone].all(), f"{what}: {(~ok[alone]).any(-1).sum()} of {alone.sum()} rows"


def test_sum_of_weights_of_zero_values():
    """2^25 tokens whose values are zero, all but the first 64 of them 12 bits
    above those in score: nothing of the result moves the reference, and the
    sum of the weights has to stay finite.  One workgroup adds up 2^20 terms in
    a lane, each sum rounded: lse is off by 2^20 * 2^-24 (and its own 2^-18)."""
    say("zero values")
    tb, group, n, r = 64, 128, 64, 8
    rec = hkv.alloc_records(1, 2, "int4", tb, 1, device=DEV)[0]
    k, v = torch.zeros(2, 2 * tb, 1, 128, device=DEV)
    k[tb:, 0, 0] = 7.0
    hkv.append_tokens(k, v, torch.arange(2 * tb, device=DEV), rec, "int4", tb)
    blocks = 2 ** 25 // tb
    table = torch.ones(r, blocks, dtype=torch.int32, device=DEV)
    table[:, 0] = 0
    q = torch.zeros(r * n, group, 128, device=DEV, dtype=torch.bfloat16)
    q[..., 0] = 1.0
    scale = 12 * np.log(2) / 7
    out, lse = hkv.attend_records(q, rec, "int4", tb, 1, table, torch.full((r,), 2 ** 25, dtype=torch.int32, device=DEV),
                                  torch.arange(r + 1, dtype=torch.int32, device=DEV) * n, max_queries=n, causal=False,
                                  sm_scale=scale)
    torch.cuda.synchronize()
    assert (out == 0).all()
    want = np.log(64 + (2.0 ** 25 - 64) * 2.0 ** 12)
    assert torch.isfinite(lse).all()
    assert float((lse.double() - want).abs().max()) <= 2.0 ** -4 + 2.0 ** -18
