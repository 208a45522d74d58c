"""Pins of the page serving oracle, on the CPU: masks worked by hand, attention
against a softmax written out, the join against attention over all tokens."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import pages_oracle as P


@pytest.mark.parametrize("kw,want", [
    (dict(), [1, 1, 1, 1, 0, 0]),
    (dict(causal=False), [1, 1, 1, 1, 1, 1]),
    (dict(begin=2), [0, 0, 1, 1, 0, 0]),
    (dict(begin=5), [0, 0, 0, 0, 0, 0]),
    (dict(begin=5, causal=False), [0, 0, 0, 0, 0, 1]),
    (dict(window=2), [0, 0, 1, 1, 0, 0]),
    (dict(window=1, causal=False), [0, 0, 0, 1, 1, 1]),
    (dict(prefix=5), [1, 1, 1, 1, 1, 0]),
    (dict(begin=3, prefix=1), [1, 0, 0, 1, 0, 0]),
    (dict(position=0), [1, 0, 0, 0, 0, 0]),
    (dict(position=99), [1, 1, 1, 1, 1, 1]),
    (dict(position=99, window=95), [0, 0, 0, 0, 0, 1]),
    (dict(position=-1, prefix=4), [0, 0, 0, 0, 0, 0]),
], ids=str)
def test_sight_by_hand(kw, want):
    """The first of 3 queries of a request of 6 tokens: position 6 - 3 = 3."""
    assert P.sight(6, 3, 0, **kw).astype(int).tolist() == want


def test_sight_of_more_queries_than_tokens():
    """Three queries behind two tokens: the first stands before them all."""
    assert P.sight(2, 3, 0).tolist() == [False, False]
    assert P.sight(2, 3, 0, prefix=1).tolist() == [True, False]
    assert P.sight(2, 3, 1).tolist() == [True, False]
    assert P.sight(2, 3, 0, causal=False).tolist() == [True, True]


def test_attention_written_out():
    g = np.random.default_rng(1)
    k, v = g.standard_normal((2, 3, 4, 1, 128))
    q = g.standard_normal((1, 2, 128))
    table = np.array([[2, 0]], np.int32)
    slopes = np.array([0.25, -0.5])
    out, lse, *_ = P.attend_pages(q, k, v, table, [6], cap=2.0, slopes=slopes)
    rows_k, rows_v = (np.concatenate([x[2], x[0]])[:6, 0] for x in (k, v))
    for h in range(2):
        s = 2.0 * np.tanh(rows_k @ q[0, h] / np.sqrt(128) / 2.0) - slopes[h] * (5 - np.arange(6))
        p = np.exp(s)
        assert np.allclose(out[0, h], (p / p.sum()) @ rows_v, atol=1e-13)
        assert np.isclose(lse[0, h], np.log(p.sum()), atol=1e-13)


def test_join_is_attention_over_all():
    g = np.random.default_rng(2)
    k, v = g.standard_normal((2, 2, 8, 2, 128))
    q = g.standard_normal((1, 4, 128))
    whole = P.attend_pages(q, k, v, np.array([[0, 1]], np.int32), [16], causal=False)
    a = P.attend_pages(q, k, v, np.array([[0]], np.int32), [8], causal=False)
    b = P.attend_pages(q, k, v, np.array([[1]], np.int32), [8], causal=False)
    out, lse = P.join_attention(a[0], a[1], b[0], b[1])
    assert np.allclose(out, whole[0], atol=1e-13) and np.allclose(lse, whole[1], atol=1e-13)
    nothing = np.full(lse.shape, -np.inf)
    out, lse = P.join_attention(np.full(a[0].shape, np.nan), nothing, b[0], b[1])
    assert np.array_equal(out, b[0]) and np.array_equal(lse, b[1])
    out, lse = P.join_attention(np.full(a[0].shape, np.nan), nothing, b[0], nothing)
    assert (out == 0).all() and np.isneginf(lse).all()


def test_append_skips():
    pages = np.zeros((2, 3, 1, 128))
    x = np.ones((4, 1, 128)) * np.arange(1, 5)[:, None, None]
    got = P.append_pages(pages, x, [5, -1, 6, 0])
    assert got[1, 2, 0, 0] == 1 and got[0, 0, 0, 0] == 4 and got.sum() == 128 * 5
