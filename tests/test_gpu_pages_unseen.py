"""What a row of attention over pages does not see does not reach it, to the
bit: keys and values of infinities and NaN, in the very tiles that the row
walks, against the same call with finite ones in their places; at ordinary
scores and at scores whose fp32 sums depend on their order.  And what a row
does see of them it gets, in every dim and in no other."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from attend_pages_paths import CASES, ident
from oracle import pages_oracle as P
from parity_util import TORCH_OF, host_f64
from quantization_rope_reuse_amd import hkv
from test_gpu_attend_pages_paths import made as paths_made
from test_gpu_pages import DEV, dev, fresh, ints, say

pytestmark = pytest.mark.gpu
TB, H, GROUP, LEN = 16, 2, 4, 300


def made(dtype, n, seed):
    g = np.random.default_rng(seed)
    kp, vp = fresh(g, 20, TB, H, dtype)
    q = dev(g.standard_normal((n, H * GROUP, 128))).to(TORCH_OF[dtype])
    positions = np.sort(g.integers(0, LEN, n))
    return g, q, kp, vp, positions


def spoil(x, tokens, g):
    """A copy of pages with infinities and NaN in the tokens: all dims of some,
    one of others."""
    x = x.clone()
    for t in tokens:
        at = x[t // TB, t % TB]
        value = [float("nan"), float("inf"), -float("inf")][int(g.integers(3))]
        if g.random() < 0.5:
            at.fill_(value)
        else:
            at[:, int(g.integers(128))] = value
    return x


SCORES = [dict(), dict(sm_scale=30.0), dict(sm_scale=2.0 ** 20), dict(sm_scale=-2.0 ** 28), dict(cap=20.0, sm_scale=0.5),
          dict(slopes=0.5), dict(slopes=2.0 ** 24, cap=2.0 ** 30, sm_scale=2.0 ** 27)]


@pytest.mark.parametrize("scores", SCORES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", [1, 7, 70])
def test_unseen(dtype, n, scores):
    say("unseen", dtype, n, scores)
    g, q, kp, vp, positions = made(dtype, n, 31)
    scores = dict(scores)
    if "slopes" in scores:
        scores["slopes"] = torch.full((H * GROUP,), scores["slopes"], device=DEV)
    for kw in (dict(), dict(window=9), dict(window=70, prefix_len=[5])):
        pre = kw.get("prefix_len", [0])[0]
        m = np.arange(LEN)[None]
        p = positions[:, None]
        sees = ((m <= p) & (m > p - kw.get("window", LEN))) | (m < pre)
        # tokens that at most some of the rows see, among them their neighbours
        bad = np.unique(np.concatenate([positions + 1, positions - 9, g.integers(pre, LEN, 12)]))
        bad = bad[(bad >= pre) & (bad < LEN)]
        kb, vb = spoil(kp, bad[::2], g), spoil(vp, bad, g)
        fine = dev(~sees[:, bad].any(1))
        if not fine.any():
            bad = bad[bad > positions.min()]
            kb, vb = spoil(kp, bad[::2], g), spoil(vp, bad, g)
            fine = dev(~sees[:, bad].any(1))
        assert fine.any() and len(bad)
        more = dict(scores, positions=ints(positions), max_queries=n,
                    **{k: ints(v) if k == "prefix_len" else v for k, v in kw.items()})
        rest = (ints(np.arange(20)[None]), ints([LEN]), ints([0, n]))
        clean, cl = hkv.attend_pages(q, kp, vp, *rest, **more)
        out, lse = hkv.attend_pages(q, kb, vb, *rest, **more)
        assert torch.isfinite(clean.float()).all()
        assert torch.equal(out[fine], clean[fine]) and torch.equal(lse[fine], cl[fine]), kw


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", [1, 7, 70])
def test_seen(dtype, n):
    """Dim 5 of a seen token is infinite, dim 77 of another NaN, dim 100 of two
    infinite with unlike signs: those dims of the rows that see them, no others."""
    say("seen", dtype, n)
    g, q, kp, vp, positions = made(dtype, n, 32)
    at = int(np.median(positions))
    vb = vp.clone()
    for token, dim, value in ((at, 5, float("inf")), (at // 2, 77, float("nan")), (at // 3, 100, float("inf")),
                              (at, 100, -float("inf"))):
        vb[token // TB, token % TB, :, dim] = value
    rest = (ints(np.arange(20)[None]), ints([LEN]), ints([0, n]))
    more = dict(positions=ints(positions), max_queries=n, sm_scale=0.02)
    clean, cl = hkv.attend_pages(q, kp, vp, *rest, **more)
    out, lse = hkv.attend_pages(q, kp, vb, *rest, **more)
    assert torch.equal(lse, cl)
    others = [d for d in range(128) if d not in (5, 77, 100)]
    assert torch.equal(out[..., others], clean[..., others])
    for i, pos in enumerate(positions):
        assert (out[i, :, 5] == float("inf")).all() if pos >= at else torch.equal(out[i, :, 5], clean[i, :, 5])
        assert torch.isnan(out[i, :, 77]).all() if pos >= at // 2 else torch.equal(out[i, :, 77], clean[i, :, 77])
        assert torch.isnan(out[i, :, 100]).all() if pos >= at else (out[i, :, 100] == float("inf")).all() \
            if pos >= at // 3 else torch.equal(out[i, :, 100], clean[i, :, 100])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 7, 70])
def test_values_near_the_largest(dtype, n):
    """Sums of weights times values leave fp32's range before the weights' sum
    is divided out; the result does not.  Scores grow along the tokens, so that
    the reference moves often."""
    say("largest values", dtype, n)
    g, q, kp, vp, positions = made(dtype, n, 33)
    half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}[dtype]
    unit = hkv.attend_pages(q, kp, vp * 0 + 1, ints(np.arange(20)[None]), ints([LEN]), ints([0, n]), max_queries=n,
                            positions=ints(positions), slopes=torch.full((H * GROUP,), 0.7, device=DEV))
    big = 3.0e38
    out, lse = hkv.attend_pages(q, kp, vp * 0 + big, ints(np.arange(20)[None]), ints([LEN]), ints([0, n]), max_queries=n,
                                positions=ints(positions), slopes=torch.full((H * GROUP,), 0.7, device=DEV))
    assert torch.equal(lse, unit[1])
    # weights of 8, 16 or 24 bits against their sum, 300 sums in fp32, the result's rounding
    want = host_f64((torch.ones((), device=DEV) * big).to(TORCH_OF[dtype]))
    assert (np.abs(host_f64(out) / want - 1) <= 2 * half + 2.0 ** -8 * (dtype == "bf16") + 300 * 2.0 ** -24 + 2.0 ** -16).all()


@pytest.mark.parametrize("case", CASES, ids=ident)
def test_unseen_by_every_way_of_sharing_out(case):
    """Ranges, cuts and joins, with entries left out: some of each request's tokens
    not finite, rows that see none of them."""
    say("unseen, shared out", case)
    dtype, tb, h, group, lens, asks, own, share = case
    g, kp, vp, table, q_start, q, kw, _ = paths_made(case, 34)
    n = q.shape[0]
    window = max(lens) // 20
    positions = np.concatenate([np.sort(g.integers(0, max(x, 1), a)) for x, a in zip(lens, asks)]).astype(np.int64)
    kb, vb = kp.clone(), vp.clone()
    fine = np.ones(n, bool)
    for r, x in enumerate(lens):
        held = -(-x // tb)
        table[r, :held][g.random(held) < 0.1] = -1
        bad = np.unique(g.integers(0, x, 1 + x // 300)) if x else np.zeros(0, np.int64)
        for i in range(q_start[r], q_start[r + 1]):
            fine[i] = not P.sight(x, 0, 0, positions[i], 0, 2, window)[bad].any()
        for t in bad:
            page = int(table[r, t // tb])
            if page >= 0:
                vb[page, t % tb], kb[page, t % tb] = float("nan"), float("inf")
    fine = dev(fine)
    args = (ints(np.minimum(table, 2 ** 30)), ints(lens), ints(q_start))
    more = dict(max_queries=max(asks), positions=ints(positions), window=window, prefix_len=ints([2] * len(lens)))
    clean, cl = hkv.attend_pages(q, kp, vp, *args, **more)
    out, lse = hkv.attend_pages(q, kb, vb, *args, **more)
    assert torch.equal(out[fine], clean[fine]) and torch.equal(lse[fine], cl[fine])
    assert torch.isfinite(clean.float()).all()
