"""fp16 results have weights of two fp16 parts.

Scores next to zero, so that their own error does not hide the weights':
weights are then all of one size, times the values' scales.  Relative to
spread = sum p |v|, a weight of two parts is off by 2^-22, exp2 and the sums
over T tokens by 2^-20 + T * 2^-24, the scores by twice their error ds.  A
second part below fp16's normal numbers is off by 2^-25, beside a largest
weight of at least 2^12.5: 2^-37 of the largest value for every token.  Then
one rounding of the result, 2^-11.

On the CPU: weights of one part break that bound, weights of two hold it.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
from oracle import serve_oracle as S
from parity_util import TORCH_OF, host_f64
from quantization_rope_reuse_amd import hkv
from test_gpu_serve import DEV, HALF, TINY, dev, on_device, say

TB, LEN = 16, 43
SCALE = 2.0 ** -12


def inputs(fmt, n, h, group):
    g = np.random.default_rng([n, h, group])
    x = g.standard_normal((2, 3, TB, h, 128))
    rec = O.put(x[0][None], x[1][None], np.arange(3), fmt)[0][0]
    q = (1.5 * g.standard_normal((n, h * group, 128))).astype(np.float16)
    return rec, q, np.array([[2, 0, 1]], np.int32)


def bound(rec, fmt, h, want, spread, reach, moved):
    most = np.abs(O.dequant_records(rec[None], fmt, TB, h)[1]).max()
    ds = reach * (160 * 2.0 ** -24 + (2.0 ** -21 if moved else 0))
    tokens = 3 * TB
    return spread * (2.0 ** -22 + 2.0 ** -20 + tokens * 2.0 ** -24 + 2 * ds[..., None]) \
        + tokens * most * 2.0 ** -37 + np.abs(want) * HALF["f16"] + TINY["f16"]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int4", "fp8"])
@pytest.mark.parametrize("n,h,group", [(1, 2, 4), (4, 2, 4), (7, 2, 4), (110, 1, 4), (37, 1, 128)])
@pytest.mark.parametrize("moved", [False, True])
def test_fp16_results(fmt, n, h, group, moved):
    say("fp16 weights", fmt, n, h, group, moved)
    rec, q, table = inputs(fmt, n, h, group)
    kw = dict(sm_scale=SCALE, causal=False)
    dm = dict(delta_m=np.full(table.shape, 321, np.int32)) if moved else {}
    out, _ = hkv.attend_records(dev(q), on_device(rec, fmt, TB, h), fmt, TB, h, dev(table), dev(np.array([LEN], np.int32)),
                                dev(np.array([0, n], np.int32)), max_queries=n, **kw,
                                **({"delta_m": dev(dm["delta_m"])} if moved else {}))
    torch.cuda.synchronize()
    want, _, spread, reach = S.attend(q, rec, fmt, TB, h, table, [LEN], [0, n], **kw, **dm)
    tol = bound(rec, fmt, h, want, spread, reach, moved)
    err = np.abs(host_f64(out) - want)
    assert (err <= tol).all(), f"{(err > tol).sum()} of {err.size}, worst {(err / tol).max()} of the bound"


@pytest.mark.parametrize("fmt", ["int4", "fp8"])
def test_bound_sees_the_second_part(fmt):
    n, h, group = 7, 2, 4
    rec, q, table = inputs(fmt, n, h, group)
    want, _, spread, reach = S.attend(q, rec, fmt, TB, h, table, [LEN], [0, n], sm_scale=SCALE, causal=False)
    tol = bound(rec, fmt, h, want, spread, reach, False)
    k, v = (x[0][table[0]].reshape(-1, h, 128)[:LEN].astype(np.float64) for x in O.dequant_records(rec[None], fmt, TB, h))
    size = np.abs(v).max(-1, keepdims=True)                # stands for the scale: a weight's other factor
    out = {}
    for parts in (1, 2):
        got = np.empty_like(want)
        for i in range(h * group):
            s = q[:, i].astype(np.float64) @ k[:, i // group].T * SCALE
            p = np.exp(s - s.max(-1, keepdims=True))
            w = p * size[:, i // group, 0] / size.max() * 2.0 ** 13
            held = w.astype(np.float16).astype(np.float64)
            if parts == 2:
                held += (w - held).astype(np.float16)
            code = v[:, i // group] / size[:, i // group] * size.max()
            got[:, i] = held @ code / (p.sum(-1, keepdims=True) * 2.0 ** 13)
        out[parts] = np.abs(got.astype(np.float16) - want) <= tol
    assert out[2].all() and (~out[1]).mean() > 0.01
