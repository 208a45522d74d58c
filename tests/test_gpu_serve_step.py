"""The serving calls as one step: the example against a server computed by the
64-bit oracle from the same records, on another stream, and captured into a
HIP graph that is replayed on changing lengths."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest
import torch

import oracle as O  # noqa: F401
from oracle import serve_oracle as S
from conftest import ROOT
from parity_util import host_f64
from quantization_rope_reuse_amd import hkv

sys.path.insert(0, os.path.join(ROOT, "examples"))
pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("fmt", ["int4", "fp8"])
def test_example_runs_and_its_plans_hold(fmt):
    import serve_step
    print("[serve] example", fmt, flush=True)
    server, history = serve_step.run(layers=2, steps=20, fmt=fmt)
    torch.cuda.synchronize()
    # request 0 (37 + 20 tokens) ended and came back with 9; row 3 has 20 + 1
    assert server.kv_len.tolist() == [9, 5 + 20 + 2, 100 + 20 + 2, 21]
    held = [-(-n // 16) for n in server.kv_len.tolist()]
    assert int(server.free_count) == 64 - sum(held)
    used = [b for r, n in enumerate(held) for b in server.table[r, :n].tolist()]
    assert len(set(used)) == len(used) and not set(used) & set(server.free[:64 - sum(held)].tolist())
    for x, plan in history:
        assert torch.isfinite(x.float()).all() and not plan.refused.any()


def _step(q, k, v, st, out):
    """One layer's step into preallocated tensors."""
    plan = hkv.plan_step(st["len"], st["new"], st["table"], st["free"], st["count"], 16, q.shape[0], out=out["plan"])
    hkv.rope_heads(q, k, plan.positions, 1e4, "half_split", q_out=out["q"], k_out=out["k"])
    hkv.append_tokens(out["k"], v, plan.slots, st["rec"], "int4", 16)
    hkv.attend_records(out["q"], st["rec"], "int4", 16, 2, st["table"], plan.kv_len, plan.q_start, max_queries=6,
                       out=out["out"], lse=out["lse"], workspace=out["ws"])


def _state(seed):
    g = np.random.default_rng(seed)
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    lens = g.integers(1, 60, 3).astype(np.int32)
    ids = g.permutation(40).astype(np.int32)
    table = np.full((3, 24), -1, np.int32)
    held, at = -(-lens // 16), 0
    for r, n in enumerate(held):
        table[r, :n] = ids[at:at + n]
        at += n
    rec = hkv.alloc_records(1, 40, "int4", 16, 2, device=DEV)[0]
    x = torch.randn(40 * 16, 4, 128, device=DEV)
    hkv.append_tokens(x[:, :2], x[:, 2:], torch.arange(640, device=DEV), rec, "int4", 16)
    st = dict(len=d(lens), new=d(np.array([1, 6, 2], np.int32)), table=d(table), free=d(np.r_[ids[at:], ids[:at]]),
              count=d(np.array([40 - at], np.int32)), rec=rec)
    out = dict(plan=hkv.alloc_plan(3, 9, device=DEV), q=torch.empty(9, 8, 128, device=DEV, dtype=torch.bfloat16),
               k=torch.empty(9, 2, 128, device=DEV, dtype=torch.bfloat16),
               out=torch.empty(9, 8, 128, device=DEV, dtype=torch.bfloat16), lse=torch.empty(9, 8, device=DEV),
               ws=torch.empty(max(16, hkv.attend_workspace_bytes(40, 16, 2, 3, 24, 9, 8, 6, torch.bfloat16)),
                              dtype=torch.uint8, device=DEV))
    q, k, v = (torch.randn(9, h, 128, device=DEV).bfloat16() for h in (8, 2, 2))
    return st, out, q, k, v


def _clone(t):
    if isinstance(t, hkv.StepPlan):
        return hkv.StepPlan(*(x.clone() for x in t))
    return t.clone()


def test_step_against_the_oracle_on_another_stream():
    torch.manual_seed(5)
    st, out, q, k, v = _state(1)
    host = {n: t.cpu().numpy() for n, t in st.items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _step(q, k, v, st, out)
    side.synchronize()
    p = S.plan_step(host["len"], host["new"], host["table"], host["free"], host["count"][0], 16, 9)
    for name in ("kv_len", "q_start", "positions", "slots", "refused"):
        assert np.array_equal(getattr(out["plan"], name).cpu().numpy(), p[name]), name
    rec = S.append_tokens(host_f64(out["k"]), host_f64(v), p["slots"], host["rec"], "int4", 16)
    assert np.array_equal(st["rec"].cpu().numpy(), rec)
    kr = S.rope_heads(host_f64(k), p["positions"][None], [0] * 64, range(64), 1e4, "half_split")
    assert np.abs(host_f64(out["k"]) - kr).max() < 2.0 ** -8 * np.abs(kr).max()
    o, lse, spread, reach = S.attend(host_f64(out["q"]), rec, "int4", 16, 2, p["table"], p["kv_len"], p["q_start"])
    # weights rounded to fp16 and scores in fp32 (see test_gpu_serve.py), then bf16
    tol = spread * (2.0 ** -11 + 2.0 ** -16 + 320 * 2.0 ** -24 * reach[..., None]) + np.abs(o) * 2.0 ** -8
    assert (np.abs(host_f64(out["out"]) - o) <= tol).all()
    assert (np.abs(host_f64(out["lse"]) - lse) <= reach * 160 * 2.0 ** -24 + 2.0 ** -20 + np.abs(lse) * 2.0 ** -22).all()


def test_step_in_a_graph():
    """Captured once, replayed as lengths grow: each replay against the same
    step run eagerly from the same state, with other work in between."""
    torch.manual_seed(6)
    st, out, q, k, v = _state(2)
    warm = {n: t.clone() for n, t in st.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(q, k, v, warm, out)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(q, k, v, st, out)
    for i in range(6):
        print("[serve] replay", i, flush=True)
        for t in (out["out"], out["lse"], out["q"], out["plan"].slots):
            t.fill_(7)
        twin = {n: t.clone() for n, t in st.items()}
        eager = {n: (_clone(t) if n != "ws" else torch.empty_like(t)) for n, t in out.items()}
        graph.replay()
        torch.cuda.synchronize()
        _step(q, k, v, twin, eager)
        torch.cuda.synchronize()
        for n in ("q", "k", "out", "lse"):
            assert torch.equal(out[n], eager[n]), (i, n)
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
        for t in (q, k, v):
            t.normal_()
