"""Oracle of the page serving calls: append with rotation, attention over pages
with its masks, caps and biases, and the join of two attentions, in float64."""
from __future__ import annotations

import numpy as np

from .hkv_oracle import HEAD_DIM


def append_pages(pages, x, slots):
    """Copy of pages [P, T_b, H, 128] with x [n, H, 128] in its slots; slots
    outside the pool are skipped."""
    out = pages.copy()
    total = out.shape[0] * out.shape[1]
    for t, slot in enumerate(int(s) for s in slots):
        if 0 <= slot < total:
            out[slot // out.shape[1], slot % out.shape[1]] = x[t]
    return out


def sight(length, n, j, position=None, begin=0, prefix=0, window=0, causal=True):
    """Which of `length` cached tokens query j of n sees, as a truth value each."""
    m = np.arange(length, dtype=np.int64)
    if position is not None and position < 0:
        return np.zeros(length, bool)
    pos = int(length - n + j if position is None else position)
    near = m >= int(begin)
    if causal:
        near &= m <= pos
    if window:
        near &= m > pos - int(window)
    return near | (m < int(prefix))


def attend_pages(q, k_pages, v_pages, block_table, kv_len, q_start=None, max_queries=None,
                 sm_scale=HEAD_DIM ** -0.5, causal=True, positions=None, begin=None, prefix_len=None,
                 window=0, cap=0.0, slopes=None):
    """(out, lse, error, spread, lse_error) in float64; rows of no request are
    NaN.  error [n, Hq, 128] and lse_error [n, Hq]: how far fp32 scores may move
    out and lse (first order), each score off by up to
      ds_m = 160 2^-24 reach_m               128 exact products summed, scaled
           + 2^-20 min(cap, reach_m)         (capped) a tanh good to 2^-20
           + 4 2^-24 (bias_m + reach_m)      (biased) the bias and its difference
    with reach_m = |sm_scale| sum |q k_m|; spread = sum p |v|."""
    q = np.asarray(q, np.float64)
    n, hq, _ = q.shape
    pages, tb, h = k_pages.shape[:3]
    mb = block_table.shape[1]
    out = np.full(q.shape, np.nan)
    lse = np.full((n, hq), np.nan)
    error, spread, lse_error = np.zeros(q.shape), np.zeros(q.shape), np.zeros((n, hq))
    for r in range(len(kv_len)):
        a, b = (r, r + 1) if q_start is None else (min(max(int(x), 0), n) for x in q_start[r:r + 2])
        ln = min(max(int(kv_len[r]), 0), mb * tb) if pages else 0
        tok = np.arange(ln)
        entries = block_table[r, tok // tb].astype(np.int64) if ln else np.zeros(0, np.int64)
        live = (entries >= 0) & (entries < pages)
        k = np.zeros((ln, h, HEAD_DIM))
        v = np.zeros((ln, h, HEAD_DIM))
        k[live] = k_pages[entries[live], tok[live] % tb]
        v[live] = v_pages[entries[live], tok[live] % tb]
        for j in range(b - a if max_queries is None else min(b - a, max_queries)):
            i = a + j
            pos = ln - (b - a) + j if positions is None else int(positions[i])
            sees = live & sight(ln, b - a, j, None if positions is None else pos, 0 if begin is None else begin[i],
                                0 if prefix_len is None else prefix_len[r], window, causal)
            if not sees.any():
                out[i], lse[i] = 0.0, -np.inf
                continue
            far = np.abs(pos - tok[sees]).astype(np.float64)
            for head in range(hq):
                kh = head // (hq // h)
                ks, vs = k[sees, kh], v[sees, kh]
                s = ks @ q[i, head] * sm_scale
                reach = (np.abs(ks) @ np.abs(q[i, head])) * abs(sm_scale)
                ds = 160 * 2.0 ** -24 * reach
                if cap:
                    s = cap * np.tanh(s / cap)
                    ds = ds + 2.0 ** -20 * np.minimum(cap, reach)
                if slopes is not None:
                    bias = float(slopes[head]) * far
                    s = s - bias
                    ds = ds + 4 * 2.0 ** -24 * (np.abs(bias) + reach)
                top = s.max()
                if np.isneginf(top):
                    out[i, head], lse[i, head] = 0.0, -np.inf
                    continue
                p = np.exp(s - top)
                lse[i, head] = top + np.log(p.sum())
                p /= p.sum()
                # (a weight that underflows takes nothing along)
                out[i, head] = p @ vs if np.isfinite(vs).all() else \
                    np.where(p[:, None] == 0, 0.0, p[:, None] * vs).sum(0)
                spread[i, head] = p @ np.abs(vs)
                lse_error[i, head] = p @ ds
                error[i, head] = (p * ds) @ np.abs(vs) + (p @ ds) * spread[i, head]
    return out, lse, error, spread, lse_error


def join_attention(out_a, lse_a, out_b, lse_b):
    """(out, lse) of two parts; a part of lse -inf adds nothing."""
    lse = np.logaddexp(lse_a, lse_b)
    none = np.isneginf(lse)
    base = np.where(none, 0.0, lse)
    out = np.zeros(out_a.shape)
    for x, l in ((out_a, lse_a), (out_b, lse_b)):
        w = np.where(np.isneginf(l), 0.0, np.exp(l - base))[..., None]
        out += np.where(w > 0, w * np.where(w > 0, x, 0.0), 0.0)
    return out, lse
