"""Memory of calls that run on another stream than the current one: what a
call makes for itself (outputs left as None, workspaces) comes from its own
stream's pool, so that neither work queued on the current stream before the
call nor what is allocated there after it shares that memory."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from quantization_rope_reuse_amd import hkv
from test_gpu_serve import DEV, dev, pool

pytestmark = pytest.mark.gpu


def pool_stream(t):
    """The stream whose pool holds a tensor's memory."""
    at = t.data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= at < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's")


def reserved(handle):
    return sum(s["total_size"] for s in torch.cuda.memory_snapshot() if s["stream"] == handle)


def long_context():
    """One request of 9,000 tokens, whose attention needs a workspace."""
    g = np.random.default_rng(4)
    tb, h, nb = 64, 2, 141
    rec = pool(g, "int4", nb, tb, h)
    table = dev(g.permutation(nb).astype(np.int32)[None])
    n = dev(np.array([9000], np.int32))
    q = torch.from_numpy(1.5 * g.standard_normal((1, 16, 128))).to(DEV, torch.bfloat16)
    need = hkv.attend_workspace_bytes(nb, tb, h, 1, nb, 1, 16, 1, q.dtype)
    assert need > 0
    return (q, rec, "int4", tb, h, table, n), need


@pytest.mark.parametrize("handle", [False, True])
def test_made_on_the_calls_stream(handle):
    side = torch.cuda.Stream()
    s = side.cuda_stream if handle else side
    args, need = long_context()
    i = torch.zeros(3, dtype=torch.int32, device=DEV)
    table = torch.zeros(3, 4, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = reserved(side.cuda_stream)
    made = list(hkv.attend_records(*args, stream=s))
    assert reserved(side.cuda_stream) - before >= need
    made += hkv.plan_step(i, i, table, i, i[:1], 16, 5, stream=s)
    made += hkv.rope_heads(args[0], args[0][:, :2], i[:1], 1e4, "half_split", stream=s)
    assert [pool_stream(t) for t in made] == [side.cuda_stream] * len(made)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    side.synchronize()
    # on the null stream by its handle, while another is current
    with torch.cuda.stream(side):
        out, lse = hkv.attend_records(*args, stream=0)
        assert torch.cuda.current_stream() == side
    assert pool_stream(out) == pool_stream(lse) == 0
    torch.cuda.synchronize()


@pytest.mark.parametrize("handle", [False, True])
def test_current_stream_busy_with_freed_memory(handle):
    """The current stream has fills of freed blocks of the workspace's and the
    results' sizes ahead of it, behind some milliseconds of products, and
    takes such blocks again after every call."""
    args, need = long_context()
    q = args[0]
    want, want_lse = hkv.attend_records(*args)
    side = torch.cuda.Stream()
    outs = [torch.empty_like(q) for _ in range(10)]
    m = torch.randn(8192, 8192, device=DEV).bfloat16()
    torch.cuda.synchronize()

    def fill():
        for n in (need, q.numel() * 2, want_lse.numel() * 4):
            torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0xFF)
    kept = []
    for _ in range(5):
        m @ m
    for out in outs:
        fill()
        hkv.attend_records(*args, out=out, stream=side.cuda_stream if handle else side)
        kept.append(hkv.attend_records(*args, stream=side.cuda_stream if handle else side))
    fill()
    torch.cuda.synchronize()
    for out, (a, b) in zip(outs, kept):
        assert torch.equal(out, want) and torch.equal(a, want) and torch.equal(b, want_lse)


@pytest.mark.parametrize("handle", [False, True])
def test_cache_calls_make_on_their_stream(handle):
    """The same for the put with CRC, the CRC, the page order, the selection
    and the frames; results as on the current stream."""
    tb, h, nb = 64, 2, 8
    k, v = (torch.randn(1, nb, tb, h, 128, device=DEV).bfloat16() for _ in range(2))
    table = torch.arange(nb - 1, -1, -1, dtype=torch.int32, device=DEV)
    rec = hkv.alloc_records(1, nb, "fp8", tb, h, device=DEV)
    frames = hkv.alloc_frames(1, nb, "fp8", tb, h, device=DEV)
    x, y = (torch.randn(5000, 64, device=DEV) for _ in range(2))

    def calls(**kw):
        made = [hkv.quant_crc("fp8", k, v, table, rec, **kw), hkv.crc32_blocks(rec, "fp8", tb, h, **kw),
                hkv.page_visit_order(table, nb, **kw)]
        made.append(hkv.token_drift(x, y, **kw))
        made.append(hkv.select_top_tokens(made[-1], 100, **kw))
        hkv.quant_fp8(k, v, table, hkv.frame_records(frames), **kw)
        hkv.frame_headers(frames, "fp8", tb, h, made[0], table, **kw)
        made += [hkv.frame_verify(frames, "fp8", tb, h, **kw), hkv.frame_delta_m(frames, "fp8", tb, h, table, **kw)]
        return made
    want = calls()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    before = reserved(0)
    got = calls(stream=side.cuda_stream if handle else side)
    assert [pool_stream(t) for t in got] == [side.cuda_stream] * len(got)
    assert reserved(0) == before         # workspaces included
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(side):
        assert pool_stream(hkv.crc32_blocks(rec, "fp8", tb, h, stream=0)) == 0
    torch.cuda.synchronize()
