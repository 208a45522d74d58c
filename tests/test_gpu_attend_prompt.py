"""Attention over records by the prompt kernel (attend_paths.py PROMPTS, which
test_attend_share.py holds to it), with the tolerances of test_gpu_serve.py
(check_attend): causal and not, moved keys, rows of very different size, blocks
left out and slots full of NaN, the same bits again, in a graph, on another
stream."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
from attend_paths import PROMPTS, blocks_of
from parity_util import TORCH_OF
from quantization_rope_reuse_amd import hkv
from test_gpu_serve import DEV, check_attend, dev, on_device, pool, say

pytestmark = pytest.mark.gpu


def name_of(c):
    return f"{c[0]}-{c[1]}-T{c[2]}-H{c[3]}x{c[4]}-{sum(c[6])}q"


def setup(case, seed):
    fmt, dtype, tb, h, group, lens, asks, _ = case
    g = np.random.default_rng([seed, tb, h, group])
    held = [-(-n // tb) for n in lens]
    table = np.full((len(lens), blocks_of(lens, tb)), -1, np.int32)
    ids, at = g.permutation(sum(held) + 2).astype(np.int32), 0
    for r, n in enumerate(held):
        table[r, :n] = ids[at:at + n]
        at += n
    q = torch.from_numpy(1.5 * g.standard_normal((sum(asks), h * group, 128))).to(DEV, TORCH_OF[dtype])
    return g, pool(g, fmt, sum(held) + 2, tb, h), table, np.concatenate([[0], np.cumsum(asks)]), q


@pytest.mark.parametrize("case", PROMPTS, ids=name_of)
@pytest.mark.parametrize("moved", [False, True])
def test_prompts(case, moved):
    say("prompt kernel", name_of(case), moved)
    fmt, dtype, tb, h, group, lens, asks, _ = case
    g, rec, table, q_start, q = setup(case, 21)
    kw = {}
    if moved:
        dm = g.integers(-3000, 3001, table.shape).astype(np.int32)
        dm[:, 1::2] = dm[:, :1]
        kw = dict(delta_m=dm, rope_base=1e4, pairs="half_split" if tb == 64 else "interleaved")
    check_attend(q, rec, fmt, tb, h, table, lens, q_start, "causal", max_queries=max(asks), **kw)
    check_attend(q, rec, fmt, tb, h, table, lens, q_start, "all tokens", causal=False, sm_scale=-0.07, **kw)


@pytest.mark.parametrize("fmt", ["int4", "fp8"])
def test_holes_and_garbage(fmt):
    say("prompt kernel holes", fmt)
    g = np.random.default_rng(5)
    tb, h, nb, group = 16, 1, 30, 60
    rec = pool(g, fmt, nb, tb, h, garbage=True)
    lens, asks = [150, 64, 30], [40, 38, 45]               # 45 queries of 30 tokens: 15 see nothing
    table = np.full((3, 10), -1, np.int32)
    ids, at = 1 + g.permutation(nb - 1).astype(np.int32), 0
    for r, n in enumerate(lens):
        held = -(-n // tb)
        table[r, :held] = ids[at:at + held]
        at += held
        slots = table[r, np.arange(n) // tb].astype(np.int64) * tb + np.arange(n) % tb
        x = torch.from_numpy(g.standard_normal((2, n, h, 128)).astype(np.float32)).to(DEV)
        hkv.append_tokens(x[0].contiguous(), x[1].contiguous(), dev(slots), rec, fmt, tb)
    table[0, 2], table[0, 8] = -1, 2 ** 31 - 1
    table[1, :] = -5
    for dtype in ("bf16", "f32"):
        q = torch.from_numpy(g.standard_normal((sum(asks), group, 128))).to(DEV, TORCH_OF[dtype])
        check_attend(q, rec, fmt, tb, h, table, lens, np.concatenate([[0], np.cumsum(asks)]), dtype)


@pytest.mark.parametrize("dtype,sizes", [("bf16", (0, 1e-30, 1e-6, 1, 30, 1e4)), ("f32", (0, 1e-30, 1e-6, 1, 30, 1e4)),
                                         ("f16", (0, 6e-8, 1e-4, 1, 30, 1e4))])
def test_sizes_of_values(dtype, sizes):
    """Rows of zeros, tiny and large rows beside each other, values whose
    scales differ by 2^30, one token that takes all the weight."""
    say("prompt kernel sizes", dtype)
    g = np.random.default_rng(8)
    nb, tb, h, n, group = 5, 16, 1, 36, 64
    x = g.standard_normal((2, nb, tb, h, 128))
    x[0, 1] = 0.0
    x[1, 2] = 0.0
    x[1, :, 3] *= 2.0 ** 14
    x[1, :, 5] *= 2.0 ** -16
    q = g.standard_normal((n, group, 128)) * np.asarray(sizes)[g.integers(0, len(sizes), (n, group, 1))]
    q = torch.from_numpy(q).to(DEV, TORCH_OF[dtype])
    table = np.array([[2, 0, 3, 1, 4]], np.int32)
    for fmt in ("int4", "fp8"):
        rec = on_device(O.put(x[0][None], x[1][None], np.arange(nb), fmt)[0][0], fmt, tb, h)
        check_attend(q, rec, fmt, tb, h, table, [75], [0, n], f"{fmt} {dtype}", causal=False)
        check_attend(q, rec, fmt, tb, h, table, [75], [0, n], f"{fmt} {dtype} moved", causal=False,
                     delta_m=np.full(table.shape, 777, np.int32))


@pytest.mark.parametrize("case", [PROMPTS[0], PROMPTS[3], PROMPTS[4]], ids=name_of)
def test_same_bits_in_a_graph_and_on_another_stream(case):
    """Replayed with other lengths and eager work between the replays, and on
    another stream with memory of its own: the eager call's bits."""
    fmt, dtype, tb, h, group, lens, asks, _ = case
    _, rec, table, q_start, q = setup(case, 6)
    t, n, qs = dev(table), dev(np.asarray(lens, np.int32)), dev(q_start.astype(np.int32))
    need = hkv.attend_workspace_bytes(rec.shape[0], tb, h, len(lens), table.shape[1], sum(asks), h * group, max(asks),
                                      q.dtype)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)

    def call(o, s, **kw):
        return hkv.attend_records(q, rec, fmt, tb, h, t, n, q_start=qs, max_queries=max(asks), out=o, lse=s, **kw)
    call(out, lse, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, lse, workspace=ws)
    side = torch.cuda.Stream()
    for cut in (0, 1, 59, 0):
        n.copy_(dev(np.asarray(lens, np.int32) - cut))
        want, want_lse = call(None, None)
        torch.cuda.synchronize()
        out.fill_(7)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        a, b = call(None, None, stream=side)
        side.synchronize()
        assert torch.equal(a, want) and torch.equal(b, want_lse)
