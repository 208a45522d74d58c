"""Attention over pages by every way its work is shared out (the calls of
attend_pages_paths.py, whose paths test_attend_pages_share.py holds) against
the oracle in 64 bits: ranges, cuts that leave some rows whole, joins of few and
many partial results."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from attend_pages_paths import CASES, ident
from quantization_rope_reuse_amd import hkv
from test_gpu_pages import check, ints, setup

pytestmark = pytest.mark.gpu


def made(case, seed):
    """Pages, table, queries; positions of the requests' rows, in order, the first of them 0."""
    dtype, tb, h, group, lens, asks, own, share = case
    g, kp, vp, table, q_start, q = setup((dtype, tb, h, group, lens, asks, "tokens"), seed)
    positions = None
    if own:
        positions = np.concatenate([np.sort(np.append(0, 1 + g.permutation(max(n, a) - 1)[:a - 1]))
                                    for n, a in zip(lens, asks)])
    return g, kp, vp, table, q_start, q, dict(positions=positions), share[0] == "chunk"


@pytest.mark.parametrize("case", CASES, ids=ident)
def test_paths(case):
    print("paths", case, flush=True)
    lens, most = case[4], max(case[5])
    g, kp, vp, table, q_start, q, kw, one_part = made(case, 11)
    check(q, kp, vp, table, lens, q_start, "causal", one_part, max_queries=most, **kw)
    slopes = np.where(np.arange(q.shape[1]) % 2, 0.01, -0.0001)
    check(q, kp, vp, table, lens, q_start, "cap, slopes", one_part, max_queries=most, cap=9.0, slopes=slopes, **kw)
    check(q, kp, vp, table, lens, q_start, "window", one_part, max_queries=most, window=max(lens) // 3, **kw)
    n = q.shape[0]
    check(q, kp, vp, table, lens, q_start, "documents", one_part, max_queries=most, begin=g.integers(0, max(lens), n),
          prefix_len=g.integers(0, 40, len(lens)), **kw)
    check(q, kp, vp, table, lens, q_start, "all tokens", one_part, max_queries=most, causal=False)


@pytest.mark.parametrize("case", CASES, ids=ident)
def test_paths_with_holes(case):
    """Entries left out, and pages that no entry names full of NaN."""
    print("paths with holes", case, flush=True)
    dtype, tb, h, group, lens, asks, own, share = case
    g, kp, vp, table, q_start, q, kw, one_part = made(case, 12)
    named = np.zeros(kp.shape[0], bool)
    for r, n in enumerate(lens):
        held = -(-n // tb)
        out = g.random(held) < 0.3
        table[r, :held][out] = np.where(g.random(out.sum()) < 0.5, -1, kp.shape[0])
        inside = table[r, :held]
        named[inside[(inside >= 0) & (inside < kp.shape[0])]] = True
    for x in (kp, vp):
        x[torch.from_numpy(~named).to(x.device)] = float("nan")
    check(q, kp, vp, table, lens, q_start, "holes", one_part, max_queries=max(asks), **kw)


@pytest.mark.parametrize("case", CASES, ids=ident)
def test_workspace(case):
    """A workspace of just the bytes asked for, full of NaN or of what the last
    call left: the same bits, and nothing written behind it."""
    print("workspace", case, flush=True)
    dtype, tb, h, group, lens, asks, own, share = case
    _, kp, vp, table, q_start, q, kw, _ = made(case, 13)
    pos = None if kw["positions"] is None else ints(kw["positions"])
    need = hkv.attend_pages_workspace_bytes(kp.shape[0], tb, h, len(lens), table.shape[1], q.shape[0], q.shape[1],
                                            max(asks), q.dtype)
    # (sizes alone decide the bytes: another call of them may be cut where this is not)
    assert need > 0 or share in (("rows", 0, 1), ("chunk", 1))
    args = (q, kp, vp, ints(table), ints(lens), ints(q_start))
    a, la = hkv.attend_pages(*args, max_queries=max(asks), positions=pos)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device=q.device)
    for _ in range(2):
        b, lb = hkv.attend_pages(*args, max_queries=max(asks), positions=pos, workspace=ws[:need])
        assert torch.equal(a, b) and torch.equal(la, lb)
        assert (ws[need:] == 0xFF).all()


CUT = [c for c in CASES if c[-1] in (("chunk", 4), ("chunk", 3), ("rows", 112, 8)) and c[0] != "f32"]


@pytest.mark.parametrize("case", CUT, ids=ident)
def test_cut_calls_in_a_graph(case):
    """Captured once and replayed with other lengths and queries, eager work in
    between: each replay against the same call made eagerly."""
    print("cut calls in a graph", case, flush=True)
    dtype, tb, h, group, lens, asks, own, share = case
    g, kp, vp, table, q_start, q, kw, _ = made(case, 14)
    table[table == 10 ** 9] = -1
    table, starts, length = ints(table), ints(q_start), ints(lens)
    pos = None if kw["positions"] is None else ints(kw["positions"])
    need = hkv.attend_pages_workspace_bytes(kp.shape[0], tb, h, len(lens), table.shape[1], q.shape[0], q.shape[1],
                                            max(asks), q.dtype)
    ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=q.device)

    def call(out, lse, ws):
        hkv.attend_pages(q, kp, vp, table, length, starts, max_queries=max(asks), positions=pos, out=out, lse=lse,
                         workspace=ws)

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
        length.copy_(torch.from_numpy(g.integers(0, np.asarray(lens) + 1).astype(np.int32)))
        q.normal_()


def test_calls_at_once():
    """Calls of all paths under way together on two streams, each with a
    workspace of its own, give what they give alone."""
    print("calls at once", flush=True)
    calls = []
    for case in CASES:
        _, kp, vp, table, q_start, q, kw, _ = made(case, 15)
        pos = None if kw["positions"] is None else ints(kw["positions"])
        args = (q, kp, vp, ints(table), ints(case[4]), ints(q_start))
        calls.append((args, dict(max_queries=max(case[5]), positions=pos)))
    alone = []
    for args, kw in calls:
        alone.append(hkv.attend_pages(*args, **kw))
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [hkv.attend_pages(*args, **kw, stream=streams[i % 2]) for _ in range(3) for i, (args, kw) in enumerate(calls)]
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, alone[i % len(calls)][0]) and torch.equal(lse, alone[i % len(calls)][1]), CASES[i % len(calls)]


@pytest.mark.parametrize("queries", [1, 40])
def test_shared_pages(queries):
    """Requests that share pages, and a table that names a page twice."""
    print("shared pages", queries, flush=True)
    case = ("bf16", 64, 2, 4, [1500, 1400, 1300], [queries] * 3, "tokens")
    _, kp, vp, table, q_start, q = setup(case, 16)
    table[1, :9] = table[0, :9]
    table[2, 3:7] = table[2, 2]
    check(q, kp, vp, table, case[4], q_start, "shared", queries > 1, max_queries=queries)
