"""Serving calls on the GPU against the 64-bit oracle: step plans, rotary
positions with several axes, token append, attention over records, and the
four of them as one step, eager, on another stream and in a HIP graph.

Tolerances count roundings (half a step each, u = eps / 2 of the type):
* plan, append: exact.
* rope: cosine and sine within 2^-22, products and sum in fp32 (3 steps of
  2^-24 of |a| + |b|), the angle off by 2^-51 of itself; then one rounding of
  the result.
* attention, per output element, with spread = sum p |v| and reach = the
  largest sm_scale * sum |q k| (both from the oracle):
    scores are fp32 sums of 128 exact products, off by at most 160 * 2^-24 *
    reach (plus 2^-21 * reach where moved keys turn the query, rounded to 22
    bits), which moves a weight by that relative amount, in the numerator
    and the denominator; weights enter their product rounded to fp16 (2^-11)
    for 16-bit queries and to two fp16 parts (2^-22) for fp32; exp2 and the
    sums over T tokens in fp32 (2^-20 + T * 2^-24); all relative to spread;
    then one rounding of the result.  lse is off by the score's error and
    2^-20 + 2^-22 |lse|.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
from oracle import serve_oracle as S
from parity_util import TORCH_OF, host_f64
from quantization_rope_reuse_amd import hkv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}     # half the smallest subnormal


def dev(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, dtype)


def say(*a):
    print("[serve]", *a, flush=True)


# --- plan ------------------------------------------------------------------

def run_plan(kv_len, new, table, free, count, tb, n_tokens, stride=None):
    wide = np.full((table.shape[0], stride or table.shape[1]), 77, np.int32)
    wide[:, :table.shape[1]] = table
    t = dev(wide)
    f, c = dev(free), dev(np.array([count], np.int32))
    p = hkv.plan_step(dev(kv_len), dev(new), t[:, :table.shape[1]], f, c, tb, n_tokens)
    torch.cuda.synchronize()
    if stride:
        assert (t[:, table.shape[1]:] == 77).all()
    return dict(table=t[:, :table.shape[1]].cpu().numpy(), free=f.cpu().numpy(), free_count=int(p.free_count),
                kv_len=p.kv_len.cpu().numpy(), q_start=p.q_start.cpu().numpy(),
                positions=p.positions.cpu().numpy(), slots=p.slots.cpu().numpy(), refused=p.refused.cpu().numpy())


def check_plan(args, what, stride=None):
    want = S.plan_step(*args)
    got = run_plan(*args, stride=stride)
    for key, w in want.items():
        assert np.array_equal(np.asarray(got[key], np.int64), np.asarray(w, np.int64)), f"{what}: {key}"


def draw_plan(g, r, tb, mb, scarce):
    kv_len = g.integers(0, mb * tb + 1, r).astype(np.int32)
    new = g.choice([0, 1, 1, 1, 3, tb, 2 * tb + 1, -1, -5], r).astype(np.int32)
    held = -(-kv_len.astype(np.int64) // tb)
    ids = g.permutation(int(held.sum()) + r * 3 + 1).astype(np.int32)
    table = np.full((r, mb), -1, np.int32)
    table[np.arange(mb)[None] < held[:, None]] = ids[:held.sum()]
    spare = ids[held.sum():]
    count = int(g.integers(0, 4)) if scarce else spare.size
    free = np.full(ids.size, -9, np.int32)
    free[:spare.size] = spare
    return kv_len, new, table, free, count, tb, int(np.maximum(new, 0).sum()) + 5


@pytest.mark.parametrize("r,tb,mb", [(1, 16, 4), (3, 1, 7), (64, 16, 33), (65, 7, 5), (511, 64, 9), (513, 16, 3),
                                     (1500, 64, 20), (4096, 5, 6)])
@pytest.mark.parametrize("scarce", [False, True])
def test_plan(r, tb, mb, scarce):
    say("plan", r, tb, mb, scarce)
    check_plan(draw_plan(np.random.default_rng([r, tb, mb, scarce]), r, tb, mb, scarce), "plan",
               stride=mb + 3 if r % 2 else None)


def test_plan_edges():
    """No requests; no tokens; fewer token entries than tokens; a prompt over
    several workgroups; a list without room for what comes back; lengths,
    counts and entries that cannot be."""
    e = np.zeros(0, np.int32)
    check_plan((e, e, np.zeros((0, 4), np.int32), np.array([3], np.int32), 1, 16, 3), "no requests")
    check_plan((np.array([5], np.int32), np.array([0], np.int32), np.array([[2]], np.int32), np.array([3], np.int32),
                1, 16, 0), "no tokens")
    check_plan((np.array([0, 0], np.int32), np.array([9, 9], np.int32), np.full((2, 3), -1, np.int32),
                np.arange(8, dtype=np.int32), 8, 4, 11), "short arrays")
    n = 20011
    check_plan((np.array([3, 0, 70], np.int32), np.array([1, n, 1], np.int32),
                np.tile(np.arange(400, dtype=np.int32), (3, 1)), np.arange(400, dtype=np.int32), 400, 64, n + 2), "prompt")
    check_plan((np.array([40, 40], np.int32), np.array([-1, -1], np.int32),
                np.arange(20, dtype=np.int32).reshape(2, 10), np.array([7, 0, 0], np.int32), 1, 4, 1), "no room")
    big = 2 ** 31 - 1
    check_plan((np.array([-5, big, 3, 1, 2], np.int32), np.array([2, 1, big, -big - 1, big], np.int32),
                np.array([[5, 6], [-1, 8], [-7, -1], [-3, -1], [4, -1]], np.int32), np.array([-2, big, 1], np.int32), 99, 4, 9),
               "impossible values")


def test_plan_again_is_the_same():
    args = draw_plan(np.random.default_rng(9), 200, 16, 8, False)
    t, f, c = dev(args[2]), dev(args[3]), dev(np.array([args[4]], np.int32))
    k, n = dev(args[0]), dev(args[1])
    first = hkv.plan_step(k, n, t, f, c, 16, args[6])
    t1, f1 = t.clone(), f.clone()
    again = hkv.plan_step(k, n, t, f, c, 16, args[6])
    assert all(torch.equal(a, b) for a, b in zip(first, again)) and torch.equal(t, t1) and torch.equal(f, f1)


# --- rope ------------------------------------------------------------------

ORDERS = {"text": ((64,), "blocked"), "blocked": ((16, 24, 24), "blocked"), "turns": ((24, 20, 20), "interleaved"),
          "part": ((10, 11), "blocked"), "none": ((0,), "blocked")}


def check_rope(x, got, axes, pos, dtype, pairs, base, inverse, what):
    want = S.rope_heads(x, pos, list(axes.axis), list(axes.freq), base, pairs, inverse)
    first, second = O.pair_indices(pairs)
    size = np.empty_like(want)
    size[..., first] = size[..., second] = np.abs(x[..., first]) + np.abs(x[..., second])
    phi = np.zeros((x.shape[0], 64))
    for i in range(64):
        if axes.axis[i] >= 0:
            phi[:, i] = np.abs(pos[axes.axis[i]] / float(base) ** (2 * axes.freq[i] / 128))
    ang = np.empty((x.shape[0], 1, 128))
    ang[:, 0, first] = ang[:, 0, second] = phi
    tol = size * (2.0 ** -22 + 3 * 2.0 ** -24 + ang * 2.0 ** -51) + np.abs(want) * HALF[dtype] + TINY[dtype]
    tol = np.where(ang == 0, 0, tol)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.nanmax(np.abs(got - want)[bad])}"


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pairs", ["interleaved", "half_split"])
@pytest.mark.parametrize("order", list(ORDERS))
def test_rope(dtype, pairs, order):
    say("rope", dtype, pairs, order)
    sections, how = ORDERS[order]
    g = np.random.default_rng([len(order), len(pairs), len(dtype)])
    axes = hkv.rope_axes(1e4, pairs, sections, how)
    for n, hq, hk in ((1, 1, 1), (3, 5, 0), (37, 40, 8), (130, 3, 2)):
        pos = g.integers(0, 200000, (len(sections), n)).astype(np.int32)
        pos[0, 0] = 0
        if n > 2:
            pos[:, 2] = -12345
        q = torch.from_numpy(g.standard_normal((n, hq, 128))).to(DEV, TORCH_OF[dtype])
        k = torch.from_numpy(g.standard_normal((n, hk, 128))).to(DEV, TORCH_OF[dtype]) if hk else None
        for inverse in (False, True):
            qo, ko = hkv.rope_heads(q, k, dev(pos), 1e4, pairs, sections, how, inverse=inverse)
            torch.cuda.synchronize()
            check_rope(host_f64(q), host_f64(qo), axes, pos, dtype, pairs, 1e4, inverse, f"q {n}x{hq}")
            if hk:
                check_rope(host_f64(k), host_f64(ko), axes, pos, dtype, pairs, 1e4, inverse, f"k {n}x{hk}")


def test_rope_many_tokens_strided_and_in_place():
    """Rows of a fused projection, rotated in place; many tokens."""
    say("rope in place")
    g = torch.Generator(DEV).manual_seed(1)
    n, hq, hk = 4113, 32, 8
    for dtype in ("bf16", "f32"):
        qkv = torch.randn(n, hq + 2 * hk, 128, device=DEV, generator=g).to(TORCH_OF[dtype])
        before = qkv.clone()
        pos = torch.arange(n, dtype=torch.int32, device=DEV)
        q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
        hkv.rope_heads(q, k, pos, 5e5, "half_split", q_out=q, k_out=k)
        torch.cuda.synchronize()
        assert torch.equal(qkv[:, hq + hk:], before[:, hq + hk:])
        axes, hpos = hkv.rope_axes(5e5, "half_split"), pos.cpu().numpy()[None]
        rows = np.r_[0:5, 1000:1003, n - 3:n]
        check_rope(host_f64(before[rows, :hq + hk]), host_f64(qkv[rows, :hq + hk]), axes, hpos[:, rows], dtype,
                   "half_split", 5e5, False, dtype)
        back = hkv.rope_heads(q, k, pos, 5e5, "half_split", inverse=True)
        for a, b in zip(back, (before[:, :hq], before[:, hq:hq + hk])):
            assert float((a.float() - b.float()).norm() / b.float().norm()) < 3 * HALF[dtype] + 2.0 ** -21


def test_rope_keeps_what_does_not_turn():
    """Infinities and NaN of pairs without an axis, and of position 0, stay
    where they are."""
    q = torch.randn(2, 3, 128, device=DEV)
    q[:, 0, 5], q[:, 1, 127], q[:, 2, 100] = float("inf"), float("nan"), -float("inf")
    pos = torch.tensor([0, 9], dtype=torch.int32, device=DEV)
    out, _ = hkv.rope_heads(q, None, pos, 1e4, "half_split")
    assert torch.equal(out[0].view(torch.int32), q[0].view(torch.int32))
    out, _ = hkv.rope_heads(q, None, pos, 1e4, "half_split", sections=(0,))
    assert torch.equal(out.view(torch.int32), q.view(torch.int32))


# --- append ----------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["fp8", "int4"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tb,h,n", [(16, 8, 5), (1, 1, 3), (7, 3, 40), (64, 8, 700), (16, 5, 1)])
def test_append(fmt, dtype, tb, h, n):
    say("append", fmt, dtype, tb, h, n)
    g = np.random.default_rng([tb, h, n, len(fmt), len(dtype)])
    nb = -(-n // tb) + 2
    x = g.standard_normal((2, n, h, 128)) * np.exp2(g.integers(-12, 8, (2, n, h, 1)))
    x[0, 0, 0] = 0.0
    x[1, n - 1, h - 1, 1:] = 0.0
    k, v = (torch.from_numpy(a).to(DEV, TORCH_OF[dtype]) for a in x)
    slots = g.permutation(nb * tb)[:n].astype(np.int64)
    if n > 3:
        slots[1], slots[2], slots[3] = -1, nb * tb, 2 ** 62
    rec = hkv.alloc_records(1, nb, fmt, tb, h, device=DEV)[0]
    rec.copy_(dev(g.integers(0, 256, tuple(rec.shape)).astype(np.uint8)))
    want = S.append_tokens(host_f64(k), host_f64(v), slots, rec.cpu().numpy(), fmt, tb)
    hkv.append_tokens(k, v, dev(slots), rec, fmt, tb)
    torch.cuda.synchronize()
    got = rec.cpu().numpy()
    assert np.array_equal(got, want), f"{(got != want).sum()} bytes differ"


def test_append_strided_and_far():
    """Rows of a fused projection, into records whose offsets pass 2^32."""
    say("append far")
    tb, h, nb = 16, 2, 9
    rb = hkv.record_bytes("int4", tb, h)
    stride = 600 * 1024 * 1024
    buf = torch.empty((nb - 1) * stride + rb, dtype=torch.uint8, device=DEV)
    rec = buf.as_strided((nb, rb), (stride, 1))
    rec.zero_()
    qkv = torch.randn(20, 8, 128, device=DEV).to(torch.bfloat16)
    k, v = qkv[:, 4:6], qkv[:, 6:]
    slots = np.random.default_rng(5).permutation(nb * tb)[:20].astype(np.int64)
    slots[0] = nb * tb - 1
    slots[1:][slots[1:] == nb * tb - 1] = -1
    hkv.append_tokens(k, v, dev(slots), rec, "int4", tb)
    want = S.append_tokens(host_f64(k), host_f64(v), slots, np.zeros((nb, rb), np.uint8), "int4", tb)
    assert np.array_equal(rec.cpu().numpy(), want)
    # and attention reads them there
    table = np.arange(nb - 1, -1, -1, dtype=np.int32)[None]
    q = torch.randn(1, 4, 128, device=DEV).to(torch.bfloat16)
    check_attend(q, rec, "int4", tb, h, table, [nb * tb - 3], None, "far")


# --- attention -------------------------------------------------------------

def on_device(rec, fmt, tb, h):
    """Host records in a tensor whose block stride is a multiple of 16."""
    r = hkv.alloc_records(1, rec.shape[0], fmt, tb, h, device=DEV)[0]
    r.copy_(dev(rec))
    return r


def pool(g, fmt, nb, tb, h, garbage=False):
    """Records of normal values with channels and tokens of different size;
    garbage: NaN codes and scales wherever the caller does not write."""
    if garbage:
        r = hkv.alloc_records(1, nb, fmt, tb, h, device=DEV)[0]
        r.fill_(0xFF if fmt == "fp8" else 0x88)
        n, c = tb * h, 128 if fmt == "fp8" else 64
        r[:, 2 * n * c:].fill_(0xFF)
        return r
    x = g.standard_normal((2, nb, tb, h, 128)) * np.exp(0.5 * g.standard_normal((2, 1, 1, h, 128)))
    x *= np.exp2(g.integers(-3, 3, (2, nb, tb, 1, 1)))
    return on_device(O.put(x[0][None], x[1][None], np.arange(nb), fmt)[0][0], fmt, tb, h)


def check_attend(q, rec, fmt, tb, h, table, lens, q_start, what, **kw):
    dtype = {v: k for k, v in TORCH_OF.items()}[q.dtype]
    lens = np.asarray(lens, np.int32)
    qs = None if q_start is None else np.asarray(q_start, np.int32)
    out = torch.full_like(q, 123.0)
    lse = torch.full(q.shape[:2], 123.0, device=DEV)
    mq = kw.pop("max_queries", None)
    gk = dict(kw)
    dm = gk.get("delta_m")
    if dm is not None:
        gk["delta_m"] = dev(dm)
    hkv.attend_records(q, rec, fmt, tb, h, dev(table), dev(lens), None if qs is None else dev(qs), max_queries=mq,
                       out=out, lse=lse, **gk)
    torch.cuda.synchronize()
    want, wl, spread, reach = S.attend(host_f64(q), rec.cpu().numpy(), fmt, tb, h, table, lens, qs, **kw)
    got, gl = host_f64(out), host_f64(lse)
    none = np.isnan(wl)
    assert (got[none] == 123.0).all() and (gl[none] == 123.0).all(), f"{what}: rows of no request were written"
    keep = ~none
    ds = reach * (160 * 2.0 ** -24 + (2.0 ** -21 if dm is not None else 0))
    tokens = table.shape[1] * tb
    w = 2.0 ** -22 if dtype == "f32" else 2.0 ** -11
    tol = spread * (w + 2.0 ** -20 + tokens * 2.0 ** -24 + 2 * ds[..., None]) + np.abs(want) * HALF[dtype] + TINY[dtype]
    err = np.abs(got - want)
    bad = ~(err <= tol) & keep[..., None]
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} values, worst {np.nanmax(err[bad] / tol[bad])} of the bound"
    empty = np.isneginf(wl)
    assert (got[empty] == 0).all() and np.isneginf(gl[empty]).all(), f"{what}: empty rows"
    full = keep & ~empty
    lt = ds + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(full, wl, 0))
    assert (np.abs(gl[full] - wl[full]) <= lt[full]).all(), f"{what}: lse"


CASES = [   # fmt, dtype, block_tokens, kv heads, group, lens, queries per request
    ("int4", "bf16", 64, 8, 8, [1, 63, 64, 65, 300], [1, 1, 1, 1, 1]),
    ("int4", "f16", 16, 8, 4, [0, 5, 257], [1, 1, 1]),
    ("int4", "f32", 16, 2, 5, [100, 31, 33], [1, 1, 1]),
    ("fp8", "f16", 64, 8, 4, [129, 1000], [1, 1]),
    ("fp8", "bf16", 7, 3, 1, [50, 8, 7, 6], [1, 1, 1, 1]),
    ("fp8", "f32", 1, 1, 8, [40, 1], [1, 1]),
    ("int4", "bf16", 64, 1, 8, [1500], [1]),
    ("int4", "bf16", 64, 8, 4, [200, 40, 3], [5, 7, 9]),
    ("int4", "f16", 33, 2, 16, [90, 17], [2, 17]),
    ("int4", "bf16", 64, 2, 4, [400, 64], [150, 64]),
    ("int4", "f32", 16, 1, 3, [130], [70]),
    ("fp8", "f16", 16, 2, 4, [333, 0, 20], [66, 2, 30]),
    ("fp8", "bf16", 128, 4, 2, [700], [1]),
    ("int4", "f16", 32, 5, 33, [64, 97], [1, 2]),
    ("int4", "bf16", 48, 4, 7, [95, 97, 48], [1, 3, 0]),
]


def setup_attend(case, seed, garbage=False):
    fmt, dtype, tb, h, group, lens, asks = case
    g = np.random.default_rng([seed, tb, h, group])
    held = [-(-n // tb) for n in lens]
    nb, mb = sum(held) + 2, max(max(held), 1) + 1
    rec = pool(g, fmt, nb, tb, h)
    table = np.full((len(lens), mb), 10 ** 9, np.int32)      # entries past a request's end are never used
    ids = g.permutation(nb).astype(np.int32)
    at = 0
    for r, n in enumerate(held):
        table[r, :n] = ids[at:at + n]
        at += n
    q = torch.from_numpy(1.5 * g.standard_normal((sum(asks), h * group, 128))).to(DEV, TORCH_OF[dtype])
    return g, rec, table, np.concatenate([[0], np.cumsum(asks)]), q


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}-T{c[2]}-H{c[3]}x{c[4]}-{sum(c[6])}q")
def test_attend(case):
    say("attend", case)
    fmt, dtype, tb, h, group, lens, asks = case
    g, rec, table, q_start, q = setup_attend(case, 1)
    check_attend(q, rec, fmt, tb, h, table, lens, q_start, "causal", max_queries=max(asks))
    check_attend(q, rec, fmt, tb, h, table, lens, q_start, "all tokens", causal=False, sm_scale=-0.05)
    if all(a == 1 for a in asks):
        check_attend(q, rec, fmt, tb, h, table, lens, None, "one query each")


@pytest.mark.parametrize("case", [CASES[i] for i in (0, 1, 2, 4, 5, 7, 9, 11, 13)],
                         ids=lambda c: f"{c[0]}-{c[1]}-T{c[2]}-H{c[3]}x{c[4]}-{sum(c[6])}q")
@pytest.mark.parametrize("pairs", ["interleaved", "half_split"])
def test_attend_moved_keys(case, pairs):
    say("attend moved", case, pairs)
    fmt, dtype, tb, h, group, lens, asks = case
    g, rec, table, q_start, q = setup_attend(case, 2)
    dm = g.integers(-20000, 20001, table.shape).astype(np.int32)
    dm[:, ::3] = 0
    dm[:, 1::4] = dm[:, :1]
    check_attend(q, rec, fmt, tb, h, table, lens, q_start, pairs, max_queries=max(asks), delta_m=dm, rope_base=5e5,
                 pairs=pairs)


@pytest.mark.parametrize("fmt", ["int4", "fp8"])
@pytest.mark.parametrize("tb", [16, 64, 5])
def test_attend_holes_and_garbage(fmt, tb):
    """Blocks that the table leaves out in the middle, at the start and for a
    whole request; slots past a request's end hold NaN codes and scales, and
    so do blocks that no entry names."""
    say("attend holes", fmt, tb)
    g = np.random.default_rng(tb)
    h, nb = 2, 40
    rec = pool(g, fmt, nb, tb, h, garbage=True)
    lens = [3 * tb + 2, 6 * tb - 1, 2 * tb, 4 * tb + 1]
    table = np.full((4, 8), -1, np.int32)
    ids = 1 + g.permutation(nb - 1).astype(np.int32)         # block 0 stays garbage
    at = 0
    for r, n in enumerate(lens):
        held = -(-n // tb)
        table[r, :held] = ids[at:at + held]
        at += held
        slots = (table[r, np.arange(n) // tb].astype(np.int64) * tb + np.arange(n) % tb)
        x = torch.from_numpy(g.standard_normal((2, n, h, 128)).astype(np.float32)).to(DEV)
        hkv.append_tokens(x[0].contiguous(), x[1].contiguous(), dev(slots), rec, fmt, tb)
    table[0, 1] = -1
    table[1, 0], table[1, 3] = nb, 2 ** 31 - 1
    table[2, :] = -1
    table[3, 4] = -2 ** 31
    for dtype in ("bf16", "f32"):
        q = torch.from_numpy(g.standard_normal((9, 8, 128))).to(DEV, TORCH_OF[dtype])
        check_attend(q, rec, fmt, tb, h, table, lens, [0, 1, 4, 5, 9], dtype)
        dm = g.integers(-99, 99, table.shape).astype(np.int32)
        check_attend(q, rec, fmt, tb, h, table, lens, [0, 1, 4, 5, 9], dtype, delta_m=dm)


def test_attend_impossible_values():
    """Lengths and query ranges outside what the arrays hold are clamped, an
    empty pool and rows of no blocks give empty rows, and queries beyond
    max_queries are left alone."""
    say("attend impossible")
    g = np.random.default_rng(0)
    rec = pool(g, "int4", 6, 16, 2)
    table = np.arange(6, dtype=np.int32).reshape(2, 3)
    q = torch.from_numpy(g.standard_normal((6, 4, 128))).to(DEV, torch.bfloat16)
    check_attend(q, rec, "int4", 16, 2, table, [2 ** 31 - 1, -7], [0, 2, 2 ** 31 - 1], "lens")
    check_attend(q, rec, "int4", 16, 2, table, [40, 20], [-5, 3, 1], "backwards")
    check_attend(q, rec, "int4", 16, 2, table, [40, 20], [2, 3, 6], "first rows of no request")
    check_attend(q, rec[:0], "int4", 16, 2, table, [40, 20], [0, 3, 6], "no records")
    check_attend(q, rec, "int4", 16, 2, table[:, :0], [40, 20], [0, 3, 6], "no blocks")
    out, lse = torch.full_like(q, 5), torch.full((6, 4), 5.0, device=DEV)
    hkv.attend_records(q, rec, "int4", 16, 2, dev(table), dev(np.array([40, 20], np.int32)),
                       dev(np.array([0, 4, 6], np.int32)), max_queries=2, out=out, lse=lse)
    full, _ = hkv.attend_records(q, rec, "int4", 16, 2, dev(table), dev(np.array([40, 20], np.int32)),
                                 dev(np.array([0, 4, 6], np.int32)))
    torch.cuda.synchronize()
    assert torch.equal(out[[0, 1, 4, 5]], full[[0, 1, 4, 5]]) and (out[2:4] == 5).all() and (lse[2:4] == 5).all()


def test_attend_sizes_of_values():
    """Queries and scales near the ends of their types: rows of zeros, rows
    of subnormals, rows of 1e4 beside rows of 1e-30, one token that takes all
    the weight, values whose scales differ by 2^30."""
    say("attend sizes")
    g = np.random.default_rng(8)
    nb, tb, h = 4, 16, 2
    x = g.standard_normal((2, nb, tb, h, 128))
    x[0, 1] = 0.0
    x[1, 2] = 0.0
    x[1, :, 3] *= 2.0 ** 14
    x[1, :, 5] *= 2.0 ** -16
    for fmt in ("int4", "fp8"):
        rec = on_device(O.put(x[0][None], x[1][None], np.arange(nb), fmt)[0][0], fmt, tb, h)
        for dtype, sizes in (("bf16", (0, 1e-38, 1e-30, 1, 30, 1e4)), ("f32", (0, 1e-40, 1e-30, 1, 30, 1e4)),
                             ("f16", (0, 6e-8, 1e-4, 1, 30, 1e4))):
            q = np.stack([g.standard_normal((4, 128)) * s for s in sizes])
            q = torch.from_numpy(q).to(DEV, TORCH_OF[dtype])
            table = np.tile(np.array([2, 0, 3, 1], np.int32), (len(sizes), 1))
            check_attend(q, rec, fmt, tb, h, table, [59] * len(sizes), None, f"{fmt} {dtype}")
            check_attend(q, rec, fmt, tb, h, table, [59] * len(sizes), None, f"{fmt} {dtype} moved",
                         delta_m=np.full(table.shape, 777, np.int32))


def test_attend_long_and_strided():
    """A long context cut over many workgroups, queries and outputs that are
    parts of wider rows; the same call again gives the same bits."""
    say("attend long")
    g = np.random.default_rng(3)
    fmt, tb, h, nb = "int4", 64, 2, 160
    rec = pool(g, fmt, nb, tb, h)
    table = g.permutation(nb).astype(np.int32)[None]
    for dtype in ("bf16", "f16", "f32"):
        rows = torch.from_numpy(1.5 * g.standard_normal((2, 12, 128))).to(DEV, TORCH_OF[dtype])
        q = rows[:, 2:10]
        n = nb * tb - 17
        check_attend(q, rec, fmt, tb, h, table, [n], [0, 2], dtype)
        check_attend(q[:1], rec, fmt, tb, h, table, [n], None, dtype,
                     delta_m=(g.integers(-9, 9, table.shape) * 1000).astype(np.int32))
        wide = torch.full((2, 20, 128), 9.0, dtype=q.dtype, device=DEV)
        a = (q, rec, fmt, tb, h, dev(table), dev(np.array([n], np.int32)), dev(np.array([0, 2], np.int32)))
        hkv.attend_records(*a, out=wide[:, 5:13])
        one, lse = hkv.attend_records(*a)
        two, lse2 = hkv.attend_records(*a)
        torch.cuda.synchronize()
        assert torch.equal(wide[:, 5:13], one) and (wide[:, :5] == 9).all() and (wide[:, 13:] == 9).all()
        assert torch.equal(one, two) and torch.equal(lse, lse2)


@pytest.mark.parametrize("seed", range(24))
def test_attend_random(seed):
    g = np.random.default_rng([99, seed])
    fmt, dtype = str(g.choice(["int4", "fp8"])), str(g.choice(["f32", "f16", "bf16"]))
    tb, h, group = int(g.choice([1, 3, 16, 32, 64, 96])), int(g.choice([1, 2, 3, 4, 8])), int(g.choice([1, 2, 3, 4, 8, 12]))
    r = int(g.integers(1, 6))
    lens = [int(x) for x in g.integers(0, 50 * min(tb, 12) + 2, r)]
    asks = [int(x) for x in g.choice([0, 1, 1, 2, 5, 21, 40], r)]
    if sum(asks) == 0:
        asks[0] = 1
    case = (fmt, dtype, tb, h, group, lens, asks)
    say("attend random", seed, case)
    g, rec, table, q_start, q = setup_attend(case, seed + 50)
    kw = dict(causal=bool(g.integers(2)), sm_scale=float(g.choice([128 ** -0.5, 0.3, 0.0])))
    if g.integers(2):
        kw.update(delta_m=g.integers(-5000, 5000, table.shape).astype(np.int32), rope_base=1e4,
                  pairs=str(g.choice(["interleaved", "half_split"])))
    check_attend(q, rec, fmt, tb, h, table, lens, q_start, str(case), **kw)
