"""The example, every call of it held to the 64-bit oracle as it runs: step
plans and appended records exactly, rotations and attention within the bounds
of test_gpu_serve.py."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest
import torch

from oracle import serve_oracle as S
from conftest import ROOT
from parity_util import host_f64
from quantization_rope_reuse_amd import hkv
from test_gpu_serve import HALF, TINY, check_rope, say

sys.path.insert(0, os.path.join(ROOT, "examples"))
pytestmark = pytest.mark.gpu


def host(t):
    return t.cpu().numpy()


class Checked:
    """The library's calls, each against the oracle."""

    def __init__(self):
        self.calls = dict(plan=0, rope=0, append=0, attend=0)

    def __getattr__(self, name):
        return getattr(hkv, name)

    def plan_step(self, kv_len, new, table, free, count, tb, n):
        want = S.plan_step(host(kv_len), host(new), host(table), host(free), int(count), tb, n)
        plan = hkv.plan_step(kv_len, new, table, free, count, tb, n)
        assert np.array_equal(host(table), want["table"]) and np.array_equal(host(free), want["free"])
        assert int(plan.free_count) == want["free_count"]
        for key in ("kv_len", "q_start", "positions", "slots", "refused"):
            assert np.array_equal(host(getattr(plan, key)), want[key]), key
        self.calls["plan"] += 1
        return plan

    def rope_heads(self, q, k, positions, base, pairs, **kw):
        before = [host_f64(x) for x in (q, k)]
        hkv.rope_heads(q, k, positions, base, pairs, **kw)
        for x, y in zip(before, (q, k)):
            check_rope(x, host_f64(y), hkv.rope_axes(base, pairs), host(positions)[None], "bf16", pairs, base, False, "rope")
        self.calls["rope"] += 1

    def append_tokens(self, k, v, slots, records, fmt, tb):
        want = S.append_tokens(host_f64(k), host_f64(v), host(slots), host(records), fmt, tb)
        hkv.append_tokens(k, v, slots, records, fmt, tb)
        assert np.array_equal(host(records), want)
        self.calls["append"] += 1

    def attend_records(self, q, records, fmt, tb, h, table, kv_len, q_start, max_queries, out):
        hkv.attend_records(q, records, fmt, tb, h, table, kv_len, q_start, max_queries=max_queries, out=out)
        want, lse, spread, reach = S.attend(host_f64(q), host(records), fmt, tb, h, host(table), host(kv_len), host(q_start))
        got, none = host_f64(out), np.isnan(lse)
        assert (got[none] == 0).all()                    # padding rows keep the example's zeros
        ds = reach * 160 * 2.0 ** -24
        tol = spread * (2.0 ** -11 + 2.0 ** -20 + table.shape[1] * tb * 2.0 ** -24 + 2 * ds[..., None]) \
            + np.abs(want) * HALF["bf16"] + TINY["bf16"]
        assert (np.abs(got - want) <= tol)[~none].all()
        self.calls["attend"] += 1


@pytest.mark.parametrize("fmt", ["int4", "fp8"])
def test_example_against_the_oracle(fmt, monkeypatch):
    import serve_step
    say("example against the oracle", fmt)
    checked = Checked()
    monkeypatch.setattr(serve_step, "hkv", checked)
    serve_step.run(layers=2, steps=6, fmt=fmt)
    assert checked.calls == dict(plan=9, rope=18, append=18, attend=18)
