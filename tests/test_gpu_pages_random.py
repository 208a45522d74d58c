"""Random calls of attention over pages, seeded: sizes, types, layouts, lengths
and masks drawn together, tokens that no row sees full of what is not finite,
against the 64-bit oracle with test_gpu_pages.py's tolerances; and appended
pages against the oracle's."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import pages_oracle as P
from parity_util import TORCH_OF, host_f64
from quantization_rope_reuse_amd import hkv
from test_gpu_pages import check, dev, fresh, ints, say

pytestmark = pytest.mark.gpu


def takes_chunk_kernel(tb, h, r, mb, mq, n, hq):
    """The rule of csrc/attend_pages_share.h: whether weights have one part."""
    group, most = hq // h, min(mq, n)
    few = n * group < 64 * r
    small = n * group < 256 * r and mb * tb <= 1024 and n * group * h * mb * tb < 10_000_000
    return most * group >= 64 and not ((few or small) and most * hq * r <= 1 << 19)


def draw(seed):
    g = np.random.default_rng([77, seed])
    dtype = ["bf16", "f16", "f32"][seed % 3]
    tb, h = int(g.choice([1, 5, 8, 16, 24, 64])), int(g.choice([1, 2, 3, 8]))
    group = int(g.choice([1, 2, 4, 7, 16]))
    r = int(g.integers(1, 9))
    longest = int(np.exp(g.uniform(0, np.log(900))))
    lens = g.integers(0, longest + 1, r)
    most = int(g.choice([1, 3, 12, 60, 150]))
    asks = g.integers(0, most + 1, r)
    while asks.sum() * h * group > 6000:                 # (the oracle goes row by row)
        asks = asks // 2
    if not asks.sum():
        asks[0] = 1
    return g, dtype, tb, h, group, lens, asks


@pytest.mark.parametrize("seed", range(60))
def test_attend(seed):
    g, dtype, tb, h, group, lens, asks = draw(seed)
    r, n = len(lens), int(asks.sum())
    held = -(-lens // tb)
    nb, mb = int(held.sum()) + 2, max(int(held.max()), 1) + int(g.integers(0, 3))
    kp, vp = fresh(g, nb, tb, h, dtype, ["tokens", "heads"][int(g.integers(2))])
    table = np.full((r, mb), -1, np.int32)
    table[np.arange(mb)[None] < held[:, None]] = g.permutation(nb)[:held.sum()]
    if g.random() < 0.3:
        table[g.random(table.shape) < 0.15] = nb
    start = np.concatenate([[0], np.cumsum(asks)])
    wide = dev(g.standard_normal((n, h * group + 3, 128))).to(TORCH_OF[dtype])
    q = wide[:, 1:1 + h * group]
    top = max(int(lens.max()), 1)
    kw = dict(sm_scale=float(g.choice([128 ** -0.5, 0.3, -0.02])), causal=bool(g.random() < 0.7))
    if g.random() < 0.5:
        kw["positions"] = g.integers(-2, top + 3, n)
    if g.random() < 0.4:
        kw["window"] = int(g.integers(1, top + 2))
    if g.random() < 0.4:
        kw["begin"] = g.integers(-1, top, n)
    if g.random() < 0.4:
        kw["prefix_len"] = g.integers(0, top // 2 + 2, r)
    if g.random() < 0.3:
        kw["cap"] = float(g.choice([1.0, 15.0]))
    if g.random() < 0.3:
        kw["slopes"] = g.standard_normal(h * group) * 0.05
    mq = int(asks.max()) + int(g.integers(0, 3))
    say("random", seed, dtype, tb, h, group, lens.tolist(), asks.tolist(), sorted(kw))
    # what no row sees holds what is not finite
    seen = np.zeros((nb, tb), bool)
    for i in range(r):
        m = np.arange(lens[i])
        any_row = np.zeros(lens[i], bool)
        for j in range(asks[i]):
            at = start[i] + j
            any_row |= P.sight(lens[i], asks[i], j, None if "positions" not in kw else kw["positions"][at],
                               kw["begin"][at] if "begin" in kw else 0, kw["prefix_len"][i] if "prefix_len" in kw else 0,
                               kw.get("window", 0), kw["causal"])
        page = table[i, m // tb]
        live = any_row & (page >= 0) & (page < nb)
        seen[page[live], m[live] % tb] = True
    unseen = dev(~seen)
    kp[unseen], vp[unseen] = float("inf"), float("nan")
    out, _ = check(q, kp, vp, table, lens.tolist(), start, "random", takes_chunk_kernel(tb, h, r, mb, mq, n, h * group),
                   max_queries=mq, **kw)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("seed", range(24))
def test_append(seed):
    g, dtype, tb, h, group, lens, asks = draw(1000 + seed)
    n, page_dtype = int(g.integers(1, 300)), ["bf16", "f16", "f32"][int(g.integers(3))]
    nb = -(-n // tb) + int(g.integers(0, 4))
    say("random append", seed, dtype, page_dtype, n, tb, h)
    kp, vp = fresh(g, nb, tb, h, page_dtype, ["tokens", "heads"][int(g.integers(2))])
    before = [host_f64(x) for x in (kp, vp)]
    wide = dev(g.standard_normal((n, 2 * h + 1, 128))).to(TORCH_OF[dtype])
    k, v = wide[:, 1:1 + h], wide[:, 1 + h:]
    slots = g.permutation(nb * tb)[:n].astype(np.int64)
    slots[g.random(n) < 0.1] = int(g.choice([-1, nb * tb, 2 ** 62]))
    pos = g.integers(-100, 10 ** 6, n)
    pairs = ["half_split", "interleaved"][int(g.integers(2))]
    turned = hkv.rope_heads(k.float(), None, ints(pos), 1e4, pairs)[0].to(TORCH_OF[page_dtype])
    hkv.append_pages(k, v, dev(slots), kp, vp, positions=ints(pos), rope_base=1e4, pairs=pairs)
    for got, old, x in zip((kp, vp), before, (turned, v.to(TORCH_OF[page_dtype]))):
        assert np.array_equal(host_f64(got), P.append_pages(old, host_f64(x), slots))
