"""The page serving calls as they are used together: a step on pages (plan,
append, attend) on another stream and in a HIP graph replayed on changing
lengths, a context fetched from records with some of its tokens recomputed, and
attention over records joined with attention over pages."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import pages_oracle as P
from oracle import serve_oracle as S
from parity_util import host_f64
from quantization_rope_reuse_amd import hkv
from test_gpu_pages import DEV, check, dev, ints, say

pytestmark = pytest.mark.gpu
TB, HQ, H, MOST = 16, 8, 2, 9


def _state(seed, dtype=torch.bfloat16):
    g = np.random.default_rng(seed)
    lens = g.integers(1, 60, 3).astype(np.int32)
    ids = g.permutation(40).astype(np.int32)
    table = np.full((3, 24), -1, np.int32)
    held, at = -(-lens // TB), 0
    for r, n in enumerate(held):
        table[r, :n] = ids[at:at + n]
        at += n
    kp, vp = torch.randn(2, 40, TB, H, 128, device=DEV).to(dtype)
    st = dict(len=dev(lens), new=dev(np.array([1, 6, 2], np.int32)), table=dev(table), free=dev(np.r_[ids[at:], ids[:at]]),
              count=dev(np.array([40 - at], np.int32)), k=kp, v=vp)
    bytes_ = hkv.attend_pages_workspace_bytes(40, TB, H, 3, 24, MOST, HQ, 6, dtype)
    out = dict(plan=hkv.alloc_plan(3, MOST, device=DEV), q=torch.empty(MOST, HQ, 128, device=DEV, dtype=dtype),
               out=torch.empty(MOST, HQ, 128, device=DEV, dtype=dtype), lse=torch.empty(MOST, HQ, device=DEV),
               ws=torch.empty(max(16, bytes_), dtype=torch.uint8, device=DEV))
    return st, out, torch.randn(MOST, HQ + 2 * H, 128, device=DEV).to(dtype)


def _step(qkv, st, out, **scores):
    """One layer's step into preallocated tensors."""
    q, k, v = qkv.split([HQ, H, H], 1)
    plan = hkv.plan_step(st["len"], st["new"], st["table"], st["free"], st["count"], TB, MOST, out=out["plan"])
    hkv.append_pages(k, v, plan.slots, st["k"], st["v"], positions=plan.positions, rope_base=1e4, q=q, q_out=out["q"])
    hkv.attend_pages(out["q"], st["k"], st["v"], st["table"], plan.kv_len, plan.q_start, max_queries=6, out=out["out"],
                     lse=out["lse"], workspace=out["ws"], **scores)


def _clone(t):
    return hkv.StepPlan(*(x.clone() for x in t)) if isinstance(t, hkv.StepPlan) else t.clone()


def test_step_against_the_oracle_on_another_stream():
    say("step on another stream")
    torch.manual_seed(5)
    st, out, qkv = _state(1)
    host = {n: t.cpu().numpy() if t.dtype != torch.bfloat16 else host_f64(t) for n, t in st.items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _step(qkv, st, out)
    side.synchronize()
    p = S.plan_step(host["len"], host["new"], host["table"], host["free"], host["count"][0], TB, MOST)
    turned = hkv.rope_heads(qkv[:, :HQ], qkv[:, HQ:HQ + H], out["plan"].positions, 1e4, "half_split")
    assert torch.equal(out["q"], turned[0])
    for page, before, x in ((st["k"], host["k"], turned[1]), (st["v"], host["v"], qkv[:, HQ + H:])):
        assert np.array_equal(host_f64(page), P.append_pages(before, host_f64(x), p["slots"]))
    eager, lse = check(out["q"], st["k"], st["v"], p["table"], p["kv_len"].tolist(), p["q_start"], "step", max_queries=6)
    n = int(p["q_start"][-1])
    assert torch.equal(out["out"][:n], eager[:n]) and torch.equal(out["lse"][:n], lse[:n])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_step_in_a_graph(dtype):
    """Captured once, replayed as lengths grow: each replay against the same
    step run eagerly from the same state, with other work in between; a second
    graph that shares the workspace is replayed in turn."""
    torch.manual_seed(6)
    st, out, qkv = _state(2, dtype)
    scores = dict(window=50, cap=30.0, prefix_len=ints([2, 0, 1]))
    warm = {n: t.clone() for n, t in st.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(qkv, warm, out, **scores)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(qkv, st, out, **scores)
    o2, l2 = torch.empty_like(out["out"]), torch.empty_like(out["lse"])
    with torch.cuda.graph(other):
        hkv.attend_pages(out["q"], st["k"], st["v"], st["table"], out["plan"].kv_len, out["plan"].q_start, max_queries=6,
                         out=o2, lse=l2, workspace=out["ws"], causal=False)
    for i in range(6):
        say("replay", i)
        for t in (out["out"], out["lse"], out["q"], out["plan"].slots, o2, l2):
            t.fill_(7)
        twin = {n: t.clone() for n, t in st.items()}
        eager = {n: (_clone(t) if n != "ws" else torch.empty_like(t)) for n, t in out.items()}
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        _step(qkv, twin, eager, **scores)
        free, fl = hkv.attend_pages(eager["q"], twin["k"], twin["v"], twin["table"], eager["plan"].kv_len,
                                    eager["plan"].q_start, max_queries=6, causal=False, out=torch.full_like(o2, 7),
                                    lse=torch.full_like(l2, 7))
        torch.cuda.synchronize()
        for n in ("q", "out", "lse"):
            assert torch.equal(out[n], eager[n]), (i, n)
        assert torch.equal(o2, free) and torch.equal(l2, fl), i
        for a, b in zip(out["plan"], eager["plan"]):
            assert torch.equal(a, b), i
        for n in st:
            assert torch.equal(st[n], twin[n]), (i, n)
        assert torch.isfinite(out["out"].float()).all()
        # the next step's inputs
        st["len"].copy_(out["plan"].kv_len)
        st["count"].copy_(out["plan"].free_count)
        st["new"].copy_(torch.tensor([[1, 1, 1], [6, 2, 1], [-1, 3, 0], [4, 0, 5], [2, 2, 2], [1, 1, 1]][i],
                                     dtype=torch.int32))
        qkv.normal_()


def test_many_rows_in_a_graph():
    """The kernel for many rows and its join, captured, replayed with other
    lengths, positions and contents."""
    say("many rows in a graph")
    torch.manual_seed(8)
    n, tb, mb = 300, 16, 128
    kp, vp = torch.randn(2, 2 * mb, tb, H, 128, device=DEV).half()
    table = torch.randperm(2 * mb, device=DEV).int().view(2, mb)
    q = torch.randn(n, HQ, 128, device=DEV).half()
    lens, q_start, pos = ints([2000, 700]), ints([0, 180, n]), torch.arange(n, device=DEV).int()
    ws = torch.empty(hkv.attend_pages_workspace_bytes(2 * mb, tb, H, 2, mb, n, HQ, n, torch.half), dtype=torch.uint8,
                     device=DEV)
    assert ws.numel() > 16                       # partial results are joined
    out, lse = torch.empty_like(q), torch.empty(n, HQ, device=DEV)

    def call(out, lse, ws):
        hkv.attend_pages(q, kp, vp, table, lens, q_start, positions=pos, out=out, lse=lse, workspace=ws)

    call(out, lse, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, lse, ws)
    for i in range(4):
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        eager, el = torch.empty_like(out), torch.empty_like(lse)
        call(eager, el, torch.empty_like(ws))
        assert torch.equal(out, eager) and torch.equal(lse, el), i
        lens.copy_(torch.randint(1, 2048, (2,)))
        q_start.copy_(torch.tensor([0, int(torch.randint(1, n, ())), n]))
        pos.copy_(torch.randint(-3, 2048, (n,)))
        q.normal_()


def test_recomputed_tokens_of_a_fetched_context():
    """A context of two cached chunks, fetched from FP8 records into pages at
    new positions; the tokens that drifted most are recomputed: their new keys
    and values replace the fetched ones and their queries attend at their own
    positions."""
    say("recompute")
    torch.manual_seed(9)
    g = np.random.default_rng(9)
    nb, n = 12, 12 * TB
    rec = hkv.alloc_records(1, nb, "fp8", TB, H, device=DEV)
    old = torch.randn(2, nb, TB, H, 128, device=DEV).bfloat16()
    order = torch.arange(nb, dtype=torch.int32, device=DEV)
    hkv.quant_fp8(old[0], old[1], order, rec)
    kp, vp = torch.zeros(2, 20, TB, H, 128, device=DEV).bfloat16()
    table = ints(g.permutation(20)[:nb])
    delta = ints(np.where(np.arange(nb) < 6, 96, -96))
    hkv.fetch_dequant_rope_shift(rec, "fp8", table, delta, 1e4, "half_split", kp, vp)
    cached = torch.randn(n, 256, device=DEV)
    fresh = cached + torch.rand(n, 1, device=DEV) * torch.randn(n, 256, device=DEV)
    picked = hkv.select_top_tokens(hkv.token_drift(cached, fresh), 28)
    x = torch.randn(28, HQ + 2 * H, 128, device=DEV).bfloat16()
    q, k, v = x.split([HQ, H, H], 1)
    slots = table.long()[picked.long() // TB] * TB + picked % TB
    before = kp.clone()
    q = hkv.append_pages(k, v, slots, kp, vp, positions=picked, rope_base=1e4, q=q)
    assert int((kp != before).any(-1).any(-1).sum()) == 28
    check(q, kp, vp, table.cpu().numpy()[None], [n], [0, 28], "recompute", positions=picked.cpu().numpy())


@pytest.mark.parametrize("fmt", ["int4", "fp8"])
def test_records_joined_with_pages(fmt):
    """A cache whose older tokens are records and whose newer ones lie in pages:
    attention over each, joined, against the 64-bit oracles joined."""
    say("joined", fmt)
    torch.manual_seed(10)
    cold, hot, asks = [100, 0, 33], [20, 7, 5], [3, 1, 2]
    rec = hkv.alloc_records(1, 12, fmt, TB, H, device=DEV)[0]
    x = torch.randn(12 * TB, 2 * H, 128, device=DEV).bfloat16()
    hkv.append_tokens(x[:, :H], x[:, H:], torch.arange(12 * TB, device=DEV), rec, fmt, TB)
    kp, vp = torch.randn(2, 8, TB, H, 128, device=DEV).bfloat16()
    ct, ht = ints(np.arange(24).reshape(3, 8) % 12), ints([[5, 1], [7, -1], [0, -1]])
    q = torch.randn(6, HQ, 128, device=DEV).bfloat16()
    q_start = ints([0, 3, 4, 6])
    a, la = hkv.attend_records(q, rec, fmt, TB, H, ct, ints(cold), q_start, max_queries=3, causal=False)
    b, lb = hkv.attend_pages(q, kp, vp, ht, ints(hot), q_start, max_queries=3)
    out, lse = hkv.join_attention(a, la, b, lb)
    wa, wla, spread_a, reach_a = S.attend(host_f64(q), rec.cpu().numpy(), fmt, TB, H, ct.cpu().numpy(), cold, q_start.cpu().numpy(),
                           causal=False)
    wb, wlb, error_b, spread_b, _ = P.attend_pages(host_f64(q), host_f64(kp), host_f64(vp), ht.cpu().numpy(), hot, q_start.cpu().numpy())
    want, wl = P.join_attention(wa, wla, wb, wlb)
    # Each part is rounded to bf16 (2^-8 of it) and weighted by at most 1; the
    # records' weights enter their product with 11 bits and their scores are
    # off by 160 2^-24 reach, both of which count against sum p |v| (spread),
    # which may be far above |part|; the pages' part has 16 bits and its own
    # error; then the join's weights (2^-18) and the result's rounding.
    parts = np.abs(wa) + np.abs(wb)
    tol = parts * (2.0 ** -8 + 2.0 ** -18) + spread_a * (2.0 ** -11 + 2.0 ** -16 + 320 * 2.0 ** -24 * reach_a[..., None]) \
        + spread_b * 2.0 ** -15 + 2 * error_b + np.abs(want) * 2.0 ** -8
    assert (np.abs(host_f64(out) - want) <= tol).all()
    assert (np.abs(host_f64(lse) - wl) <= 2.0 ** -14 + 2.0 ** -14 * np.abs(wl)).all()
    # (request 1 has nothing cold)
    assert torch.equal(out[3], b[3])
