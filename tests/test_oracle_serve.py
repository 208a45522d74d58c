"""Pins of the serving oracle, on the CPU: step plans worked by hand, the
rotation against the one-axis oracle and against differences, the append
against the put, attention against a softmax written out."""
from __future__ import annotations

import numpy as np
import pytest

import oracle as O
from oracle import serve_oracle as S

I = np.int32


def test_plan_by_hand():
    """Blocks of 4 tokens, rows of 3: request 0 decodes inside a block, 1
    crosses into a new one, 2 ends and returns two blocks, 3 starts with 5
    tokens, 4 is too long for its row."""
    table = np.array([[9, -1, -1], [4, -1, -1], [2, 3, -1], [-1, -1, -1], [7, 8, 6]], I)
    free = np.array([10, 11, 12, -5, -5, -5, -5], I)
    p = S.plan_step(np.array([1, 4, 7, 0, 11], I), np.array([1, 1, -1, 5, 2], I), table, free, 3, 4, 12)
    assert p["free"].tolist() == [10, 11, 12, 2, 3, -5, -5]
    assert p["free_count"] == 2
    assert p["table"].tolist() == [[9, -1, -1], [4, 3, -1], [2, 3, -1], [2, 12, -1], [7, 8, 6]]
    assert p["kv_len"].tolist() == [2, 5, 0, 5, 11]
    assert p["refused"].tolist() == [0, 0, 0, 0, 1]
    assert p["q_start"].tolist() == [0, 1, 2, 2, 7, 9]
    assert p["positions"].tolist() == [1, 4, 0, 1, 2, 3, 4, 11, 12, 0, 0, 0]
    assert p["slots"].tolist() == [37, 12, 8, 9, 10, 11, 48, -1, -1, -1, -1, -1]


def test_plan_runs_out_of_blocks():
    """Three requests want 1, 2 and 1 blocks of 2 free: the second and every
    later one that needs a block is refused; one that needs none goes on."""
    table = np.full((4, 4), -1, I)
    table[3, 0] = 5
    p = S.plan_step(np.array([0, 0, 0, 1], I), np.array([2, 3, 1, 1], I), table, np.array([8, 9], I), 2, 2, 7)
    assert p["refused"].tolist() == [0, 1, 1, 0]
    assert p["free_count"] == 1
    assert p["kv_len"].tolist() == [2, 0, 0, 2]
    assert p["slots"].tolist() == [18, 19, -1, -1, -1, -1, 11]


@pytest.mark.parametrize("pairs", ["interleaved", "half_split"])
def test_one_axis_is_rope(pairs):
    x = np.random.default_rng(0).standard_normal((5, 2, 128))
    pos = np.array([0, 1, 7, 100, 70000])
    got = S.rope_heads(x, pos[None], [0] * 64, range(64), 1e4, pairs)
    assert np.allclose(got, O.rope_apply(x, pos, 1e4, pairs), rtol=0, atol=1e-9)
    back = S.rope_heads(got, pos[None], [0] * 64, range(64), 1e4, pairs, inverse=True)
    assert np.allclose(back, x, rtol=0, atol=1e-12)


def test_inverse_is_the_gradient():
    """Differences of sum(w * rope(x)) against rope(w, inverse)."""
    g = np.random.default_rng(1)
    x, w = g.standard_normal((2, 3, 1, 128))
    pos = g.integers(0, 50, (3, 3))
    axis = [0] * 16 + [1] * 24 + [2] * 20 + [-1] * 4
    f = lambda y: float((w * S.rope_heads(y, pos, axis, range(64), 100.0, "half_split")).sum())  # noqa: E731
    grad = S.rope_heads(w, pos, axis, range(64), 100.0, "half_split", inverse=True)
    for t, d in ((0, 0), (1, 63), (2, 64), (0, 100), (1, 127)):
        h = np.zeros_like(x)
        h[t, 0, d] = 1e-3
        assert abs((f(x + h) - f(x - h)) / 2e-3 - grad[t, 0, d]) < 1e-9


@pytest.mark.parametrize("fmt", ["fp8", "int4"])
def test_append_is_the_put(fmt):
    g = np.random.default_rng(2)
    k, v = g.standard_normal((2, 2, 4, 3, 128)).astype(np.float32)      # [2 blocks, 4 tokens, 3 heads]
    want, _ = O.put(k[None], v[None], np.arange(2), fmt)
    rec = np.full_like(want[0], 0xAA)
    got = S.append_tokens(k.reshape(8, 3, 128), v.reshape(8, 3, 128), np.arange(8), rec, fmt, 4)
    assert np.array_equal(got, want[0])
    part = S.append_tokens(k[1, 2:3], v[1, 2:3], np.array([6]), want[0], fmt, 4)
    assert np.array_equal(part, want[0])
    assert np.array_equal(S.append_tokens(k[0], v[0], np.array([-1, 8, 99, -7]), want[0], fmt, 4), want[0])


def test_attend_written_out():
    g = np.random.default_rng(3)
    k, v = g.standard_normal((2, 3, 4, 1, 128)).astype(np.float32)
    rec, _ = O.put(k[None], v[None], np.arange(3), "fp8")
    kd, vd = (x[0].reshape(12, 128) for x in O.dequant_records(rec, "fp8", 4, 1))
    table = np.array([[2, 0, -1], [1, -1, 0]], I)
    q = g.standard_normal((4, 2, 128))
    out, lse, _, _ = S.attend(q, rec[0], "fp8", 4, 1, table, np.array([6, 10], I), np.array([0, 3, 4], I), 0.1)
    # request 0: tokens in blocks 2 and 0, queries at positions 3, 4, 5
    order = [8, 9, 10, 11, 0, 1]
    for j in range(3):
        s = kd[order[:4 + j]] @ q[j, 1] * 0.1
        p = np.exp(s) / np.exp(s).sum()
        assert np.allclose(out[j, 1], p @ vd[order[:4 + j]]) and np.isclose(lse[j, 1], np.log(np.exp(s).sum()))
    # request 1: its second block has no record
    order = [4, 5, 6, 7, 0, 1]
    s = kd[order] @ q[3, 0] * 0.1
    assert np.allclose(out[3, 0], np.exp(s) @ vd[order] / np.exp(s).sum())
    # a query before the first token sees nothing
    out, lse, _, _ = S.attend(q, rec[0], "fp8", 4, 1, table[:1], np.array([2], I), np.array([0, 4], I))
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.isfinite(lse[2:]).all()


@pytest.mark.parametrize("pairs", ["interleaved", "half_split"])
def test_shifted_keys_are_fetched_keys(pairs):
    g = np.random.default_rng(4)
    k, v = g.standard_normal((2, 2, 4, 1, 128)).astype(np.float32)
    rec, _ = O.put(k[None], v[None], np.arange(2), "int4")
    dm = np.array([[5, -300]], I)
    kr, vd = O.fetch_exact(rec, "int4", 4, 1, dm[0], 1e4, pairs)
    q = g.standard_normal((1, 1, 128))
    out, _, _, _ = S.attend(q, rec[0], "int4", 4, 1, np.array([[0, 1]], I), np.array([7], I), delta_m=dm,
                            rope_base=1e4, pairs=pairs)
    s = kr[0].reshape(8, 128)[:7] @ q[0, 0] / np.sqrt(128)
    assert np.allclose(out[0, 0], np.exp(s) @ vd[0].reshape(8, 128)[:7] / np.exp(s).sum(), atol=1e-6)
