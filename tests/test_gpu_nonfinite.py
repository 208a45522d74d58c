"""Attention over records where a query, a key or a value is not finite: what
does not see it keeps the bounds of test_gpu_serve.py (check_attend), what
does gets NaN.  (Added to those bounds: weights below 2^-126 of the largest,
which fp32 does not hold, times the largest value.)"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
from oracle import serve_oracle as S
from parity_util import TORCH_OF, host_f64
from quantization_rope_reuse_amd import hkv
from test_gpu_serve import DEV, HALF, TINY, dev, pool, say

pytestmark = pytest.mark.gpu


def compare(q, rec, fmt, tb, h, table, lens, q_start, finite, what, **kw):
    """The rows `finite` [n, heads] (None: all) against the oracle; NaN of the
    oracle have to be NaN."""
    dtype = {v: k for k, v in TORCH_OF.items()}[q.dtype]
    gk = dict(kw)
    if "delta_m" in gk:
        gk["delta_m"] = dev(gk["delta_m"])
    out, lse = hkv.attend_records(q, rec, fmt, tb, h, dev(table), dev(np.asarray(lens, np.int32)),
                                  dev(np.asarray(q_start, np.int32)),
                                  max_queries=int(np.diff(q_start).max()), **gk)
    torch.cuda.synchronize()
    x = host_f64(q)
    if finite is None:
        finite = np.ones(x.shape[:2], bool)
    x[~finite] = 0
    want, wl, spread, reach = S.attend(x, rec.cpu().numpy(), fmt, tb, h, table, lens, q_start, **kw)
    got, gl = host_f64(out), host_f64(lse)
    most = np.nanmax(np.abs(O.dequant_records(rec.cpu().numpy()[None], fmt, tb, h)[1]))
    ds = reach * (160 * 2.0 ** -24 + (2.0 ** -21 if "delta_m" in kw else 0))
    w = 2.0 ** -22 if dtype == "f32" else 2.0 ** -11
    tol = spread * (w + 2.0 ** -20 + table.shape[1] * tb * 2.0 ** -24 + 2 * ds[..., None]) \
        + np.abs(want) * HALF[dtype] + TINY[dtype] + 2.0 ** -126 * table.shape[1] * tb * most
    ok = np.where(np.isnan(want), np.isnan(got), np.abs(got - want) <= tol)
    assert ok[finite].all(), f"{what}: {(~ok[finite]).sum()} of {ok[finite].size} values"
    lt = ds + 2.0 ** -20 + 2.0 ** -22 * np.abs(wl)
    same = np.isneginf(wl) & np.isneginf(gl)
    with np.errstate(invalid="ignore"):
        ok = np.where(np.isnan(wl), np.isnan(gl), same | (np.abs(gl - wl) <= lt))
    assert ok[finite].all(), f"{what}: lse"
    return got, gl, want


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f16"])
@pytest.mark.parametrize("n,group", [(1, 4), (7, 4), (110, 4), (37, 128)])
@pytest.mark.parametrize("moved", [False, True])
@pytest.mark.parametrize("what", ["inf", "nan"])
def test_other_rows_keep_their_precision(dtype, n, group, moved, what):
    """One element of a row infinite or NaN, beside rows of 1e-6, 1e-3 and 1e5
    (4e4 in fp16): one query's 4 heads, 28 rows of a key head, 440, 4,736."""
    say("nonfinite query", dtype, n, group, moved, what)
    g = np.random.default_rng(n)
    fmt, tb, h, nb = "int4", 16, 1, 8
    rec = pool(g, fmt, nb, tb, h)
    table = g.permutation(nb).astype(np.int32)[None]
    size = np.asarray((1e-6, 1e-3, 4e4 if dtype == "f16" else 1e5))[g.integers(0, 3, (n, group))]
    x = np.clip(g.standard_normal((n, group, 128)), -1.5, 1.5) * size[..., None]
    x[n // 2, 2, 17] = np.inf if what == "inf" else np.nan
    q = torch.from_numpy(x).to(DEV, TORCH_OF[dtype])
    finite = np.ones((n, group), bool)
    finite[n // 2, 2] = False
    kw = dict(delta_m=np.full(table.shape, 777, np.int32)) if moved else {}
    for scale in (1e-5, 1.0, 1e5):
        got, _, _ = compare(q, rec, fmt, tb, h, table, [nb * tb - 3], [0, n], finite, f"scale {scale}", causal=False,
                            sm_scale=scale, **kw)
        if what == "nan":
            assert np.isnan(got[n // 2, 2]).all()


@pytest.mark.parametrize("fmt", ["int4", "fp8"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,h,group,room", [(110, 1, 4, 150), (9, 2, 4, 150), (2, 8, 2, 150), (37, 1, 128, 150),
                                            (2, 8, 4, 4200)])       # the last: two heads share a score tile
@pytest.mark.parametrize("tb", [64, 16, 7])
def test_nan_of_appended_tokens(fmt, dtype, n, h, group, room, tb):
    """Appended keys and values with a NaN element: rows that may not see the
    token yet and other heads are as without it, the rest are NaN."""
    say("nan appended", fmt, dtype, n, h, group, room, tb)
    g = np.random.default_rng([n, h, tb])
    length = 150
    nb = -(-length // tb) + 1
    rec = hkv.alloc_records(1, nb, fmt, tb, h, device=DEV)[0]
    rec.zero_()
    table = np.full((1, max(-(-room // tb), nb)), -1, np.int32)
    table[0, :nb] = g.permutation(nb)
    slots = table[0, np.arange(length) // tb].astype(np.int64) * tb + np.arange(length) % tb
    kv = g.standard_normal((2, length, h, 128))
    at_k, at_v = length - n // 2 - 1, length - 1
    kv[0, at_k, 0, 3] = np.nan
    kv[1, at_v, h - 1, 100] = np.nan
    k, v = (torch.from_numpy(a).to(DEV, TORCH_OF[dtype]) for a in kv)
    hkv.append_tokens(k, v, dev(slots), rec, fmt, tb)
    if fmt == "fp8":                     # NaN shows in the scales alone
        assert not ((rec[:, :2 * tb * h * 128] & 127) == 127).any()
    q = torch.from_numpy(g.standard_normal((n, h * group, 128))).to(DEV, TORCH_OF[dtype])
    _, _, want = compare(q, rec, fmt, tb, h, table, [length], [0, n], None, "causal")
    bad = np.isnan(want).any(-1)
    assert bad.any() and not bad[:n - n // 2 - 1].any()
    dm = np.full(table.shape, -50, np.int32)
    compare(q, rec, fmt, tb, h, table, [length], [0, n], None, "moved", delta_m=dm)
