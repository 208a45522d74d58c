"""Attention over pages whose scores are so large that fp32 holds no fraction
of them, with a cap and with a bias as without, up to the ends of fp32's range:
the token that leads takes all, and a row's only token gives its value.

Queries and keys have one element, so that the products are exact and the
leading token is known.  Tolerances: a row's one token of any weight has its
value as result, but for the weight's rounding to what its product takes (fp32
none; one part of the type where there are many rows, two parts where few), some
four roundings of 2^-24 (exponential, product, quotient, its product: 2^-20 in all)
and the result's.  lse is s off by the roundings of the scale, the product (or
cap, or slope and distance: one more each), the sum with the reference, log2(e),
ln(2) and the product with it: 8 * 2^-24 |s|."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from parity_util import TORCH_OF, host_f64
from quantization_rope_reuse_amd import hkv
from test_gpu_pages import DEV, HALF, TINY, check, dev, ints, say, setup

pytestmark = pytest.mark.gpu


def made(dtype, n, tokens, weights):
    """A request whose token m has the key weights[m] in one element, values
    of their own, and n queries of 1 there."""
    g = np.random.default_rng([n, tokens])
    kp = torch.zeros(tokens, 1, 1, 128, dtype=TORCH_OF[dtype], device=DEV)
    kp[:, 0, 0, 3] = dev(np.asarray(weights, np.float64)).to(TORCH_OF[dtype])
    vp = dev(g.standard_normal((tokens, 1, 1, 128))).to(TORCH_OF[dtype])
    q = torch.zeros(n, 1, 128, dtype=TORCH_OF[dtype], device=DEV)
    q[:, 0, 3] = 1
    return q, kp, vp, ints(np.arange(tokens)[None]), ints([tokens]), ints([0, n])


def weight_bits(dtype, n):
    """What rounding weights moves: see above."""
    one = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
    return one if n == MANY else one * one


def held(dtype, out, lse, vp, token, score):
    want = host_f64(vp)[token, 0, 0]
    tol = np.abs(want) * (weight_bits(dtype, out.shape[0]) + 2.0 ** -20 + HALF[dtype]) + TINY[dtype]
    assert (np.abs(host_f64(out)[:, 0] - want) <= tol).all(), score
    assert (np.abs(host_f64(lse) - score) <= 8 * 2.0 ** -24 * abs(score)).all(), score


# scores in log2 units around 2^16 (where references count as far), 2^24 (whole
# numbers pass fp32's step), 2^26 .. 2^28 (they pass the offset of fp16's weights)
FAR = [2.0 ** p * f for p in (15, 16, 20, 23, 24, 25, 26, 27, 28, 30, 40, 99) for f in (1.0, 1.3, 1.7)]
MANY = 300
ROWS = [3, MANY]               # the rows and the chunk kernel


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("kind", ["plain", "cap", "slopes of 0", "cap, slopes of 0"])
def test_one_token(dtype, n, kind):
    say("one token", dtype, n, kind)
    zero = torch.zeros(1, device=DEV)
    for s in FAR:
        for sign in (1, -1):
            q, kp, vp, *rest = made(dtype, n, 1, [sign])
            # a cap far above the score leaves it as it is
            cap = min(s * 2.0 ** 30, 2.0 ** 100) if "cap" in kind else None
            if cap and cap < s * 2.0 ** 14:
                continue
            out, lse = hkv.attend_pages(q, kp, vp, *rest, max_queries=n, causal=False, sm_scale=s, cap=cap,
                                        slopes=zero if "slopes" in kind else None)
            held(dtype, out, lse, vp, 0, sign * s)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_capped(dtype, n, sign):
    """Scores at their cap: every token's is the same, far as it is, so that the
    result is the mean of the values: 64 products and sums in fp32, weights as
    above."""
    say("at the cap", dtype, n, sign)
    q, kp, vp, *rest = made(dtype, n, 64, [sign] * 64)
    want = host_f64(vp)[:, 0, 0].mean(0)
    spread = np.abs(host_f64(vp)[:, 0, 0]).mean(0)
    tol = spread * (weight_bits(dtype, n) + 2.0 ** -17) + np.abs(want) * HALF[dtype] + TINY[dtype]
    for cap in (c for c in FAR if c < 2.0 ** 80):
        out, lse = hkv.attend_pages(q, kp, vp, *rest, max_queries=n, causal=False, sm_scale=cap * 2.0 ** 10, cap=cap)
        assert (np.abs(host_f64(out)[:, 0] - want) <= tol).all(), cap
        assert (np.abs(host_f64(lse) - (sign * cap + np.log(64))) <= 8 * 2.0 ** -24 * cap + 2.0 ** -20).all(), cap


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", ROWS)
def test_leading_token(dtype, n):
    """Among tokens whose scores lie a 64th of the largest apart, far more than
    a score's error, the first takes all: by products, and by the bias alone."""
    say("leading token", dtype, n)
    weights = 1 - np.arange(40) / 64
    for s in FAR[3:]:
        q, kp, vp, *rest = made(dtype, n, 40, weights)
        for kw in (dict(), dict(slopes=torch.zeros(1, device=DEV)), dict(cap=s * 2.0 ** 12) if s < 2.0 ** 80 else dict()):
            out, lse = hkv.attend_pages(q, kp, vp, *rest, max_queries=n, causal=False, sm_scale=s, **kw)
            held(dtype, out, lse, vp, 0, s)
        # the nearest token leads: all rows stand at 50, token 39 is 11 away
        out, lse = hkv.attend_pages(q, kp, vp, *rest, max_queries=n, sm_scale=0.0, positions=ints([50] * n),
                                    slopes=torch.full((1,), s, device=DEV))
        held(dtype, out, lse, vp, 39, -11 * float(np.float32(s)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("score", [1.9e38, 2.05e38, 2.15e38, 2.3e38])
def test_ends_of_the_range(dtype, n, score):
    """Scores that fp32 holds times log2(e), 3.4e38 at most: a row whose scores
    all lie at the lower end is not an empty one."""
    say("ends", dtype, n, score)
    q, kp, vp, *rest = made(dtype, n, 1, [1])
    for sign in (1, -1):
        q.fill_(0)
        q[:, 0, 3] = 2.0 ** 60 * sign
        kp.fill_(0)
        kp[0, 0, 0, 3] = 2.0 ** 40
        out, lse = hkv.attend_pages(q, kp, vp, *rest, max_queries=n, causal=False, sm_scale=score / 2.0 ** 100)
        held(dtype, out, lse, vp, 0, sign * score)
    # by the bias: one token, one before the rows
    out, lse = hkv.attend_pages(q, kp, vp, *rest, max_queries=n, sm_scale=0.0, positions=ints([1] * n),
                                slopes=torch.full((1,), score, device=DEV))
    held(dtype, out, lse, vp, 0, -float(np.float32(score)))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", [4, 70])
def test_positions_near_the_largest(dtype, n):
    """Rows at positions up to 2^31 - 1 that see a prefix, or all of it, with a
    bias by their distance: against the oracle, as in test_gpu_pages.py."""
    say("far positions", dtype, n)
    case = (dtype, 16, 2, 4, [200, 90], [n, n // 2], "tokens")
    g, kp, vp, table, q_start, q = setup(case, 51)
    positions = 2 ** 31 - 1 - g.integers(0, 300, q.shape[0])
    for slope in (1e-7, 1e-6, -1e-6):
        for kw in (dict(window=40, prefix_len=[150, 33]), dict(), dict(causal=False, cap=20.0)):
            check(q, kp, vp, table, [200, 90], q_start, "far positions", n == 70, max_queries=n, positions=positions,
                  slopes=np.full(8, slope), **kw)
