"""Angles of a whole number of quarter turns.  Of rope_base 5179020.05 pair 1
turns by half a quarter turn a position, exactly in double: at position 4 its
sine is 0 and its cosine -1.  (Of 2275.746 pair 2 does, the same with its own
index halved.)"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from quantization_rope_reuse_amd import hkv
from test_gpu_serve import DEV, check_attend, check_rope, dev, say
from parity_util import TORCH_OF, host_f64

pytestmark = pytest.mark.gpu
BASES = (5179020.0526367, 2275.74604308932)


@pytest.mark.parametrize("base", BASES)
@pytest.mark.parametrize("pairs", ["interleaved", "half_split"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rope_of_whole_quarters(base, pairs, dtype):
    say("quarters", base, pairs, dtype)
    pos = np.arange(-20, 21, dtype=np.int32)[None]
    q = torch.randn(pos.size, 3, 128, device=DEV).to(TORCH_OF[dtype])
    axes = hkv.rope_axes(base, pairs)
    for inverse in (False, True):
        out, _ = hkv.rope_heads(q, None, dev(pos), base, pairs, inverse=inverse)
        check_rope(host_f64(q), host_f64(out), axes, pos, dtype, pairs, base, inverse, "quarters")


@pytest.mark.parametrize("base", BASES)
@pytest.mark.parametrize("n,group", [(2, 4), (110, 4), (37, 128)])
def test_attend_moved_by_whole_quarters(base, n, group):
    """Records of keys that live in pairs 1 and 2 alone, moved by 4 positions;
    few rows and a prompt's."""
    say("attend quarters", base, n, group)
    g = np.random.default_rng(3)
    tb, h = 16, 1
    rec = hkv.alloc_records(1, 3, "fp8", tb, h, device=DEV)[0]
    x = g.standard_normal((2, 48, h, 128))
    x[0, :, :, [i for i in range(128) if i % 64 not in (1, 2)]] = 0
    k, v = (torch.from_numpy(a).to(DEV, torch.float32) for a in x)
    hkv.append_tokens(k, v, torch.arange(48, device=DEV), rec, "fp8", tb)
    q = torch.from_numpy(g.standard_normal((n, group, 128))).to(DEV, torch.float32)
    table = np.array([[2, 0, 1]], np.int32)
    for move in (4, -4, 12, 2):
        check_attend(q, rec, "fp8", tb, h, table, [45], [0, n], f"moved {move}", causal=False, rope_base=base,
                     delta_m=np.full(table.shape, move, np.int32), pairs="half_split")
