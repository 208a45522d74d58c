"""Attention over the longest cache that the calls take, 2^31 - 16 tokens: 511
table entries of one page whose tokens are one (a stride of 0).  All weights are
1 and all values 1, so that every sum is a whole number of less than 25 bits in
each lane, the result is 1 but for the join's roundings and the result's (2^-7
covers both), and lse the logarithm of how many tokens a row sees, in fp32: 2^-20 +
2^-22 of it."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from parity_util import TORCH_OF
from quantization_rope_reuse_amd import hkv
from test_gpu_pages import DEV, ints, say

pytestmark = pytest.mark.gpu
PAGES, TB = 511, 4202512
LEN = PAGES * TB


@pytest.mark.parametrize("dtype,n", [("bf16", 1), ("f32", 2), ("bf16", 300)])
@pytest.mark.parametrize("prefix,window,seen", [(2 ** 31 - 1, 0, LEN), (LEN, 7, LEN), (LEN - 3, 1, LEN - 2), (5, 9, 14),
                                                (0, 0, LEN)])
def test_longest(dtype, n, prefix, window, seen):
    say("longest", dtype, n, prefix, window)
    assert LEN == 2 ** 31 - 16
    k = torch.zeros(1, 1, 1, 128, dtype=TORCH_OF[dtype], device=DEV).expand(1, TB, 1, 128)
    v = torch.ones(1, 1, 1, 128, dtype=TORCH_OF[dtype], device=DEV).expand(1, TB, 1, 128)
    q = torch.ones(n, 1, 128, dtype=TORCH_OF[dtype], device=DEV)
    out, lse = hkv.attend_pages(q, k, v, torch.zeros(1, PAGES, dtype=torch.int32, device=DEV), ints([LEN]), ints([0, n]),
                                max_queries=n, window=window, prefix_len=ints([prefix]), positions=ints([LEN - 1] * n))
    torch.cuda.synchronize()
    assert ((out.float() - 1).abs() <= 2.0 ** -7).all()
    want = np.log(seen)
    assert (np.abs(lse.cpu().double().numpy() - want) <= 2.0 ** -20 + 2.0 ** -22 * want).all()
