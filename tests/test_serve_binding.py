"""The Python side of the serving calls, on the CPU."""
from __future__ import annotations

from quantization_rope_reuse_amd import hkv


def test_rope_axes_are_the_callers_own():
    """A structure that a caller changes is not what later calls get."""
    a = hkv.rope_axes(1e4, "half_split", (16, 24, 24))
    a.axis[0], a.freq[5], a.n_axes = 2, 99, 8
    b = hkv.rope_axes(1e4, "half_split", (16, 24, 24))
    assert b.axis[0] == 0 and b.freq[5] == 5 and b.n_axes == 3
    address, kept = hkv._axes_address(1e4, "half_split", (16, 24, 24), "blocked", None)
    assert kept.axis[0] == 0 and kept.freq[5] == 5
    assert hkv._axes_address(1e4, "half_split", (16, 24, 24), "blocked", None)[0] == address


def test_rope_axes_take_lists():
    assert list(hkv.rope_axes(1e4, "half_split", [1, 2], freq=[3] * 64).axis)[:4] == [0, 1, 1, -1]
    assert list(hkv.rope_axes(1e4, "half_split", order=[1, -1] * 32).axis) == [1, -1] * 32
