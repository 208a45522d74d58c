"""The native part of the binding: what it takes for a stream and a base, and
the interpreter's lock, which no library call holds."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from quantization_rope_reuse_amd import hkv
from test_gpu_serve import DEV

pytestmark = pytest.mark.gpu


def arguments():
    """Small arguments of each native call, by name."""
    i = torch.zeros(2, dtype=torch.int32, device=DEV)
    t = torch.zeros(2, 4, dtype=torch.int32, device=DEV)
    x = torch.randn(2, 2, 128, device=DEV).bfloat16()
    rec = hkv.alloc_records(1, 2, "int4", 16, 2, device=DEV)
    rec.zero_()
    pages = [torch.zeros(2, 16, 2, 128, device=DEV) for _ in range(2)]
    order = torch.arange(2, dtype=torch.int32, device=DEV)
    return {
        "hkv_plan_step": (hkv.plan_step, (i, i, t, i, i[:1], 16, 3)),
        "hkv_rope_heads": (hkv.rope_heads, (x, x, i, 1e4, "half_split")),
        "hkv_append_tokens": (hkv.append_tokens, (x, x, order.long(), rec[0], "int4", 16)),
        "hkv_attend_records": (hkv.attend_records, (x, rec[0], "int4", 16, 2, t, i)),
        "hkv_fetch_dequant_rope_shift": (hkv.fetch_dequant_rope_shift, (rec, "int4", order, i, 1e4, "half_split", *pages)),
        "hkv_fetch_dequant_rope_shift_tokens":
            (hkv.fetch_dequant_rope_shift_tokens,
             (rec, "int4", order, torch.zeros(2, 16, dtype=torch.int32, device=DEV), 1e4, "half_split", *pages)),
    }


@pytest.mark.parametrize("call", list(hkv.NATIVE_CALLS[:4] + hkv.NATIVE_CALLS[5:7]))
def test_stream_handles(call):
    """A torch stream, or its handle as any whole number, numpy's among them."""
    f, args = arguments()[call]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (None, 0, np.uint64(0), side, side.cuda_stream, np.uint64(side.cuda_stream), np.int64(side.cuda_stream)):
        f(*args, stream=s)
        torch.cuda.synchronize()
    for s in ("side", 1.5, object()):
        with pytest.raises((TypeError, ValueError)):
            f(*args, stream=s)


def test_fetch_takes_what_float_takes():
    """rope_base as a tensor, a numpy number or text, as the call always did."""
    f, args = arguments()["hkv_fetch_dequant_rope_shift"]
    for base in (torch.tensor(1e4), np.float32(1e4), "1e4", 10000):
        f(*args[:4], base, *args[5:])
    torch.cuda.synchronize()

@pytest.mark.parametrize("call", list(hkv.NATIVE_CALLS[:4] + hkv.NATIVE_CALLS[5:7]))
def test_calls_release_the_interpreter(call):
    """PyGILState_Check in the library call's place: 1, an unknown status, if
    the calling thread holds the lock."""
    f, args = arguments()[call]
    at = {n: ctypes.cast(getattr(hkv.lib(), n), ctypes.c_void_p).value for n in hkv.NATIVE_CALLS}
    check = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value
    try:
        hkv.native().bind({**at, call: check})
        f(*args)
    finally:
        hkv.native().bind(at)
