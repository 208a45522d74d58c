"""Attention over records where the work is shared out in other ways than in
the small cases: many requests, few rows and long contexts, prompts of more
than one workgroup of rows, tokens cut between workgroups, rows of very
different size beside each other; and the Python calls' refusals.  Tolerances
are those of test_gpu_serve.py (check_attend)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
from quantization_rope_reuse_amd import hkv
from test_gpu_serve import DEV, check_attend, dev, on_device, pool, say
from parity_util import TORCH_OF

pytestmark = pytest.mark.gpu


def setup(seed, fmt, dtype, tb, h, group, lens, asks, scale=1.5):
    g = np.random.default_rng(seed)
    held = [-(-n // tb) for n in lens]
    nb, mb = sum(held) + 2, max(held) + 1
    table = np.full((len(lens), mb), -1, np.int32)
    ids, at = g.permutation(nb).astype(np.int32), 0
    for r, n in enumerate(held):
        table[r, :n] = ids[at:at + n]
        at += n
    q = torch.from_numpy(scale * g.standard_normal((sum(asks), h * group, 128))).to(DEV, TORCH_OF[dtype])
    return g, pool(g, fmt, nb, tb, h), table, np.concatenate([[0], np.cumsum(asks)]), q


@pytest.mark.parametrize("n", [63, 64, 65, 200, 1025])
def test_many_requests(n):
    """Requests on both sides of what a wave's lanes hold and of what is dealt
    out evenly; some have no queries, some no tokens, one is long."""
    say("many requests", n)
    g = np.random.default_rng(n)
    lens = [int(x) for x in g.integers(0, 20, n)]
    lens[n // 2] = 1300
    asks = [int(x) for x in g.choice([0, 1, 1, 1], n)]
    asks[n // 2] = 1
    _, rec, table, q_start, q = setup(n, "int4", "bf16", 32, 2, 2, lens, asks)
    check_attend(q, rec, "int4", 32, 2, table, lens, q_start, f"{n} requests", max_queries=1)


@pytest.mark.parametrize("fmt,dtype,tb,h,group,lens,asks", [
    ("int4", "f16", 64, 2, 8, [2100], [1]),            # two heads in a score tile, ranges
    ("int4", "f32", 16, 2, 4, [1500, 40], [2, 1]),
    ("fp8", "bf16", 8, 3, 5, [900, 700], [3, 1]),       # odd heads, blocks of a run of 8
    ("fp8", "f16", 5, 2, 6, [700], [5]),                # 30 rows of a head, blocks of 5
    ("int4", "bf16", 32, 1, 12, [1100, 1], [4, 1]),     # 48 rows of a head
    ("int4", "bf16", 64, 4, 1, [5000], [1]),
], ids=str)
@pytest.mark.parametrize("moved", [False, True])
def test_ranges(fmt, dtype, tb, h, group, lens, asks, moved):
    say("ranges", fmt, dtype, tb, h, group, lens, asks, moved)
    g, rec, table, q_start, q = setup(7, fmt, dtype, tb, h, group, lens, asks)
    kw = {}
    if moved:
        dm = g.integers(-3000, 3001, table.shape).astype(np.int32)
        dm[:, 4:9] = dm[:, 4:5]
        kw = dict(delta_m=dm, rope_base=1e4, pairs="interleaved" if tb == 64 else "half_split")
    check_attend(q, rec, fmt, tb, h, table, lens, q_start, "ranges", max_queries=max(asks), **kw)


PROMPTS = [   # fmt, dtype, block_tokens, kv heads, group, lens, queries: more than 384 rows of a key head
    ("int4", "bf16", 64, 1, 4, [700, 300], [130, 100]),
    ("int4", "f16", 16, 2, 3, [200], [150]),
    ("int4", "f32", 64, 1, 5, [130], [100]),
    ("fp8", "bf16", 7, 1, 8, [90, 60, 77], [60, 0, 77]),
    ("fp8", "f16", 64, 1, 2, [1300], [200]),            # tokens cut between workgroups
    ("fp8", "f32", 32, 2, 4, [600], [97]),
]


@pytest.mark.parametrize("case", PROMPTS, ids=lambda c: f"{c[0]}-{c[1]}-T{c[2]}-H{c[3]}x{c[4]}-{sum(c[6])}q")
@pytest.mark.parametrize("moved", [False, True])
def test_prompts(case, moved):
    say("prompt", case, moved)
    fmt, dtype, tb, h, group, lens, asks = case
    g, rec, table, q_start, q = setup(11, fmt, dtype, tb, h, group, lens, asks)
    kw = {}
    if moved:
        dm = g.integers(-3000, 3001, table.shape).astype(np.int32)
        dm[:, 1::2] = dm[:, :1]
        kw = dict(delta_m=dm, rope_base=1e4, pairs="half_split" if tb == 64 else "interleaved")
    check_attend(q, rec, fmt, tb, h, table, lens, q_start, "causal", max_queries=max(asks), **kw)
    check_attend(q, rec, fmt, tb, h, table, lens, q_start, "all tokens", causal=False, sm_scale=-0.07, **kw)


@pytest.mark.parametrize("fmt", ["int4", "fp8"])
def test_prompt_holes_and_garbage(fmt):
    """A prompt over a table with blocks left out, slots past the end full of
    NaN, rows that see nothing, a request without blocks."""
    say("prompt holes", fmt)
    g = np.random.default_rng(5)
    tb, h, nb = 16, 1, 30
    rec = pool(g, fmt, nb, tb, h, garbage=True)
    lens, asks = [150, 64, 100], [110, 70, 120]            # 120 queries of 100 tokens: 20 see nothing
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
        q = torch.from_numpy(g.standard_normal((sum(asks), 4, 128))).to(DEV, TORCH_OF[dtype])
        check_attend(q, rec, fmt, tb, h, table, lens, np.concatenate([[0], np.cumsum(asks)]), dtype)


@pytest.mark.parametrize("dtype,sizes", [("bf16", (0, 1e-30, 1e-6, 1, 30, 1e4)), ("f32", (0, 1e-30, 1e-6, 1, 30, 1e4)),
                                         ("f16", (0, 6e-8, 1e-4, 1, 30, 1e4))])
def test_prompt_sizes_of_values(dtype, sizes):
    """Rows of zeros, tiny and large rows beside each other in one prompt,
    values whose scales differ by 2^30, one token that takes all the weight."""
    say("prompt sizes", dtype)
    g = np.random.default_rng(8)
    nb, tb, h, n = 5, 16, 1, 110
    x = g.standard_normal((2, nb, tb, h, 128))
    x[0, 1] = 0.0
    x[1, 2] = 0.0
    x[1, :, 3] *= 2.0 ** 14
    x[1, :, 5] *= 2.0 ** -16
    q = g.standard_normal((n, 4, 128)) * np.asarray(sizes)[g.integers(0, len(sizes), (n, 1, 1))]
    q = torch.from_numpy(q).to(DEV, TORCH_OF[dtype])
    table = np.array([[2, 0, 3, 1, 4]], np.int32)
    for fmt in ("int4", "fp8"):
        rec = on_device(O.put(x[0][None], x[1][None], np.arange(nb), fmt)[0][0], fmt, tb, h)
        check_attend(q, rec, fmt, tb, h, table, [75], [0, n], f"{fmt} {dtype}", causal=False)
        check_attend(q, rec, fmt, tb, h, table, [75], [0, n], f"{fmt} {dtype} moved", causal=False,
                     delta_m=np.full(table.shape, 777, np.int32))


def test_same_call_same_bits():
    for case in (PROMPTS[0], PROMPTS[4]):
        fmt, dtype, tb, h, group, lens, asks = case
        _, rec, table, q_start, q = setup(3, fmt, dtype, tb, h, group, lens, asks)
        a = (q, rec, fmt, tb, h, dev(table), dev(np.asarray(lens, np.int32)), dev(q_start.astype(np.int32)))
        one, two = hkv.attend_records(*a, max_queries=max(asks)), hkv.attend_records(*a, max_queries=max(asks))
        torch.cuda.synchronize()
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


@pytest.mark.parametrize("handle", [False, True])
def test_on_another_stream(handle):
    """A call on another stream than the current one, its workspace made by the
    call, while the current stream takes and fills memory of that size."""
    fmt, dtype, tb, h, group, lens, asks = "int4", "bf16", 64, 2, 8, [9000], [1]
    _, rec, table, q_start, q = setup(4, fmt, dtype, tb, h, group, lens, asks)
    t, n = dev(table), dev(np.asarray(lens, np.int32))
    want, _ = hkv.attend_records(q, rec, fmt, tb, h, t, n)
    need = hkv.attend_workspace_bytes(rec.shape[0], tb, h, 1, table.shape[1], 1, h * group, 1, q.dtype)
    assert need > 0
    side = torch.cuda.Stream()
    outs = [torch.empty_like(q) for _ in range(20)]
    lse = torch.empty(q.shape[:2], device=DEV)
    torch.cuda.synchronize()
    for out in outs:
        hkv.attend_records(q, rec, fmt, tb, h, t, n, out=out, lse=lse, stream=side.cuda_stream if handle else side)
        torch.empty(need, dtype=torch.uint8, device=DEV).fill_(0xFF)
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out, want)


def test_python_refusals():
    """Types, shapes and strides that the C calls cannot see."""
    i = torch.zeros(4, dtype=torch.int32, device=DEV)
    t = torch.zeros(4, 8, dtype=torch.int32, device=DEV)
    x = torch.zeros(4, 8, 128, dtype=torch.bfloat16, device=DEV)
    rec = hkv.alloc_records(1, 4, "fp8", 16, 8, device=DEV)[0]
    for bad in (lambda: hkv.plan_step(i, i[:3], t, i, i[:1], 16, 4), lambda: hkv.plan_step(i, i, t.T, i, i[:1], 16, 4),
                lambda: hkv.plan_step(i.long(), i, t, i, i[:1], 16, 4), lambda: hkv.plan_step(i, i, t, i, i[:1], 16, -1),
                lambda: hkv.plan_step(i, i, t, i, i[:2], 16, 4),
                lambda: hkv.rope_heads(x[..., :64], None, i, 1e4, "half_split"),
                lambda: hkv.rope_heads(x, x[:3], i, 1e4, "half_split"),
                lambda: hkv.rope_heads(x, x.float(), i, 1e4, "half_split"),
                lambda: hkv.rope_heads(x.double(), None, i, 1e4, "half_split"),
                lambda: hkv.rope_heads(x, None, i.long(), 1e4, "half_split"),
                lambda: hkv.rope_heads(x, None, i, 1e4, "half_split", sections=(16, 24, 24)),
                lambda: hkv.append_tokens(x, x, i, rec, "fp8", 16), lambda: hkv.append_tokens(x, x[:3], i.long(), rec, "fp8", 16),
                lambda: hkv.append_tokens(x, x, i.long(), rec, "fp8", 32),
                lambda: hkv.append_tokens(x, x, i.long(), rec.int(), "fp8", 16),
                lambda: hkv.attend_records(x, rec, "fp8", 16, 8, t, i[:3]),
                lambda: hkv.attend_records(x[:3], rec, "fp8", 16, 8, t, i),
                lambda: hkv.attend_records(x, rec, "fp8", 16, 8, t, i, q_start=i),
                lambda: hkv.attend_records(x, rec, "fp8", 16, 8, t, i, out=x[:3]),
                lambda: hkv.attend_records(x, rec, "fp8", 16, 8, t, i, lse=torch.zeros(4, 8, device=DEV).half()),
                lambda: hkv.attend_records(x, rec, "fp8", 16, 8, t, i, delta_m=t[:, :4]),
                lambda: hkv.attend_records(x, rec, "fp8", 16, 8, t, i, workspace=t),
                lambda: hkv.fetch_dequant_rope_shift(rec[None], "fp8", i[:3], i[:3], 1e4, "half_split",
                                                     x.new_zeros(4, 16, 8, 128), x.new_zeros(4, 16, 8, 128))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(hkv.HkvError):
        hkv.attend_records(x, rec, "fp8", 16, 8, t, i, max_queries=0)
    with pytest.raises(hkv.HkvError):
        hkv.attend_records(x[:, :7].contiguous(), rec, "fp8", 16, 8, t, i)


@pytest.mark.parametrize("case", [("int4", "bf16", 64, 2, 8, [3000], [1]), PROMPTS[0], PROMPTS[4]],
                         ids=["ranges", "prompt", "cut prompt"])
def test_in_a_graph(case):
    """Captured with a caller's workspace and replayed, with other lengths and
    eager work between the replays; each replay has the eager call's bits."""
    fmt, dtype, tb, h, group, lens, asks = case
    _, rec, table, q_start, q = setup(6, fmt, dtype, tb, h, group, lens, asks)
    t, n, qs = dev(table), dev(np.asarray(lens, np.int32)), dev(q_start.astype(np.int32))
    need = hkv.attend_workspace_bytes(rec.shape[0], tb, h, len(lens), table.shape[1], sum(asks), h * group, max(asks),
                                      q.dtype)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)

    def call(o, s):
        hkv.attend_records(q, rec, fmt, tb, h, t, n, q_start=qs, max_queries=max(asks), out=o, lse=s, workspace=ws)
    call(out, lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, lse)
    for cut in (0, 1, 60, 0):
        n.copy_(dev(np.asarray(lens, np.int32) - cut))
        want, want_lse = torch.empty_like(q), torch.empty_like(lse)
        call(want, want_lse)
        torch.cuda.synchronize()
        out.fill_(7)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_rope_gradient_against_differences():
    """<w, rope(x + e) - rope(x)> = <inverse(w), e> in fp32.  Each of the four
    results is off by 2^-22 + 3 * 2^-24 of the pair it turns (angles in double),
    each product by what it multiplies; x, e and w below 8."""
    g = torch.Generator(DEV).manual_seed(12)
    n, heads = 37, 3
    x, e, w = (torch.randn(n, heads, 128, device=DEV, generator=g) for _ in range(3))
    pos = torch.randint(0, 100000, (3, n), dtype=torch.int32, device=DEV, generator=g)
    kw = dict(sections=(24, 20, 20), order="interleaved")
    for pairs in ("interleaved", "half_split"):
        a, _ = hkv.rope_heads(x + e, None, pos, 5e5, pairs, **kw)
        b, _ = hkv.rope_heads(x, None, pos, 5e5, pairs, **kw)
        back, _ = hkv.rope_heads(w, None, pos, 5e5, pairs, inverse=True, **kw)
        step = ((x + e).double() - x.double())
        left, right = (w.double() * (a.double() - b.double())), (back.double() * step)
        bound = (2.0 ** -22 + 3 * 2.0 ** -24) * 4 * 16 * 8     # a pair's |a| + |b| <= 16, times 8
        assert abs(float((left - right).sum())) <= bound * (n * heads * 128) ** 0.5 + bound
        assert float((left.sum((1, 2)) - right.sum((1, 2))).abs().max()) <= bound * (heads * 128) ** 0.5 + bound
