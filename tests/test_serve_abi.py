"""The serving calls' argument checks, on the host: bad arguments are refused
before any HIP call (no GPU needed), empty calls launch nothing, the header is
plain C99 and every function it declares is exported."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from quantization_rope_reuse_amd import hkv as H

FAKE = 0x7F0000000000          # a 16-byte aligned address never dereferenced
HEADER = os.path.join(os.path.dirname(H.HEADER), "hkv_serve.h")


def declared():
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return sorted(set(re.findall(r"\b(hkv_[a-z0-9_]+)\s*\(", text)))


def test_exports_every_declared_symbol():
    assert declared() == ["hkv_append_tokens", "hkv_attend_records", "hkv_attend_workspace_bytes",
                          "hkv_plan_step", "hkv_rope_heads"]
    for n in declared():
        assert getattr(H.lib(), n) is not None


def test_header_is_plain_c(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("needs gcc and the ROCm headers")
    src = tmp_path / "uses.c"
    src.write_text('#include "hkv_serve.h"\nint main(void) {\n'
                   + "".join(f"  (void)&{n};\n" for n in declared())
                   + "  return hkv_plan_step(0, 0) == HKV_ERR_INVALID_ARG ? 0 : 1;\n}\n")
    pkg = os.path.dirname(H.LIB_PATH)
    exe = tmp_path / "uses"
    r = subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__",
                        "-I", "/opt/rocm/include", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe),
                        "-L", pkg, "-lhkv", f"-Wl,-rpath,{pkg}"], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    assert subprocess.run([str(exe)], timeout=60).returncode == 0


def test_struct_sizes_match_the_header(tmp_path):
    """The binding's structures against sizeof in C."""
    gcc = shutil.which("gcc")
    if gcc is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("needs gcc and the ROCm headers")
    names = {"hkv_heads": H.Heads, "hkv_step": H.Step, "hkv_rope_axes": H.RopeAxes, "hkv_requests": H.Requests,
             "hkv_key_shift": H.KeyShift}
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "hkv_serve.h"\nint main(void) {\n'
                   + "".join(f'  printf("%zu\\n", sizeof({n}));\n' for n in names) + "  return 0;\n}\n")
    exe = tmp_path / "sizes"
    subprocess.run([gcc, "-std=c99", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I",
                    os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True, timeout=120)
    sizes = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, timeout=60).stdout.split()]
    assert sizes == [ctypes.sizeof(s) for s in names.values()]


# --- plan ------------------------------------------------------------------

def _plan(**kw):
    d = dict(n_requests=4, block_tokens=16, max_blocks=8, n_tokens=32, kv_len=FAKE, new_tokens=FAKE + 64,
             block_table=FAKE + 128, table_stride=8, free_blocks=FAKE + 1024, free_capacity=64,
             free_count=FAKE + 2048, free_count_out=FAKE + 2064, kv_len_out=FAKE + 2128, q_start=FAKE + 2192,
             positions=FAKE + 4096, slots=FAKE + 8192, refused=FAKE + 16384)
    d.update(kw)
    return H.lib().hkv_plan_step(ctypes.byref(H.Step(**d)), None)


@pytest.mark.parametrize("kw", [
    dict(n_requests=-1), dict(block_tokens=0), dict(max_blocks=-1), dict(n_tokens=-1), dict(free_capacity=-1),
    dict(table_stride=7), dict(kv_len=None), dict(new_tokens=None), dict(block_table=None), dict(free_blocks=None),
    dict(free_count=None), dict(free_count_out=None), dict(free_count_out=FAKE + 2048), dict(kv_len_out=None),
    dict(kv_len_out=FAKE), dict(q_start=None), dict(positions=None), dict(slots=None), dict(refused=None),
    dict(slots=FAKE + 8196), dict(kv_len=FAKE + 2), dict(table_stride=1 << 46)], ids=str)
def test_plan_refuses(kw):
    assert _plan(**kw) == H.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(n_requests=4097), dict(max_blocks=1 << 20, block_tokens=1 << 12, table_stride=1 << 20),
                                dict(max_blocks=1 << 30, block_tokens=1, table_stride=1 << 30)], ids=str)
def test_plan_unsupported(kw):
    assert _plan(**kw) == H.ERR_UNSUPPORTED


# --- rope ------------------------------------------------------------------

def _h(heads=8, tok=1024, head=128, data=FAKE):
    return H.Heads(data, tok, head, heads)


def _rope(axes=None, pos=FAKE, axis_stride=32, n=32, q=None, k=None, qo=None, ko=None, dtype=2, **kw):
    a = H.RopeAxes.from_buffer_copy(H.rope_axes(1e4, "half_split", (16, 24, 24)))
    for f, v in kw.items():
        setattr(a, f, v)
    q, k, qo, ko = (x if x is not None else _h() for x in (q, k, qo, ko))
    return H.lib().hkv_rope_heads(None if axes is False else ctypes.byref(a), ctypes.c_void_p(pos), axis_stride, n,
                                  ctypes.byref(q), ctypes.byref(k), ctypes.byref(qo), ctypes.byref(ko), dtype, 0, None)


def _axis(i, v):
    return (ctypes.c_int8 * 64)(*[v if j == i else 0 for j in range(64)])


@pytest.mark.parametrize("kw", [
    dict(axes=False), dict(n_axes=0), dict(n_axes=9), dict(pairs=2), dict(rope_base=0.0), dict(rope_base=float("inf")),
    dict(rope_base=float("nan")), dict(axis=_axis(3, 3)), dict(axis=_axis(63, -2)),
    dict(freq=(ctypes.c_uint8 * 64)(*[128] * 64)), dict(pos=0), dict(pos=FAKE + 2), dict(axis_stride=-1), dict(n=-1),
    dict(dtype=3), dict(q=_h(7)), dict(ko=_h(9)), dict(q=_h(data=0)), dict(q=_h(data=FAKE + 8)), dict(k=_h(tok=4)),
    dict(qo=_h(head=-128)), dict(q=_h(tok=1 << 47)), dict(axis_stride=1 << 47)], ids=str)
def test_rope_refuses(kw):
    assert _rope(**kw) == H.ERR_INVALID_ARG


def test_rope_empty_and_unsupported():
    none = _h(0, data=0)
    assert _rope(n=0, pos=0) == H.OK
    assert _rope(q=none, k=none, qo=none, ko=none) == H.OK
    big = _h(1 << 24, 0, 0)
    assert _rope(q=big, qo=big) == H.ERR_UNSUPPORTED


def test_rope_axes_orders():
    a = H.rope_axes(1e4, "half_split", (2, 1, 2), "blocked")
    assert list(a.axis) == [0, 0, 1, 2, 2] + [-1] * 59 and a.n_axes == 3 and list(a.freq) == list(range(64))
    assert list(H.rope_axes(1e4, "half_split", (2, 1, 3), "interleaved").axis)[:6] == [0, 1, 2, 0, 2, 2]
    assert list(H.rope_axes(1e4, "half_split", order=tuple([1, -1] * 32)).axis) == [1, -1] * 32
    for bad in (dict(sections=(40, 40)), dict(sections=(-1, 3)), dict(order="zigzag"), dict(freq=(1, 2)),
                dict(order=(0,) * 63), dict(order=(-2,) * 64), dict(freq=(128,) * 64)):
        with pytest.raises(ValueError):
            H.rope_axes(1e4, "half_split", **bad)


# --- append and attend -----------------------------------------------------

def _shape(**kw):
    d = dict(n_layers=1, n_blocks=4, block_tokens=16, n_kv_heads=8, head_dim=128)
    d.update(kw)
    return H.Shape(**d)


def _recs(**kw):
    d = dict(base=FAKE, layer_stride_bytes=0, block_stride_bytes=33280)
    d.update(kw)
    return H.Records(**d)


def _append(shape=None, fmt=0, k=None, v=None, dtype=2, n=32, slots=FAKE, rec=None):
    shape, k, v, rec = shape or _shape(), k or _h(), v or _h(), rec or _recs()
    return H.lib().hkv_append_tokens(ctypes.byref(shape), fmt, ctypes.byref(k), ctypes.byref(v), dtype, n,
                                     ctypes.c_void_p(slots), ctypes.byref(rec), None)


@pytest.mark.parametrize("kw", [
    dict(shape=_shape(n_layers=2)), dict(shape=_shape(n_layers=0)), dict(shape=_shape(head_dim=64)),
    dict(shape=_shape(block_tokens=0)), dict(fmt=2), dict(k=_h(7)), dict(v=_h(16)), dict(dtype=5), dict(n=-1),
    dict(slots=0), dict(slots=FAKE + 4), dict(rec=_recs(base=FAKE + 8)), dict(rec=_recs(block_stride_bytes=33264)),
    dict(k=_h(data=0)), dict(v=_h(tok=1028))], ids=str)
def test_append_refuses(kw):
    assert _append(**kw) == H.ERR_INVALID_ARG


def test_append_empty():
    assert _append(n=0, slots=0) == H.OK
    assert _append(shape=_shape(n_blocks=0), slots=0) == H.OK
    assert _append(n=1 << 29, k=_h(tok=0), v=_h(tok=0)) == H.ERR_UNSUPPORTED


def _req(**kw):
    d = dict(n_requests=4, max_blocks=8, max_queries=8, block_table=FAKE, table_stride=8, kv_len=FAKE,
             q_start=FAKE)
    d.update(kw)
    return H.Requests(**d)


def _attend(shape=None, fmt=0, rec=None, req=None, q=None, dtype=2, n=32, scale=0.1, shift=None, out=None, lse=FAKE,
            ws=FAKE, ws_bytes=1 << 40):
    shape, rec, req, q, out = shape or _shape(), rec or _recs(), req or _req(), q or _h(32, 4096), out or _h(32, 4096)
    return H.lib().hkv_attend_records(
        ctypes.byref(shape), fmt, ctypes.byref(rec), ctypes.byref(req), ctypes.byref(q), dtype, n, scale, 1,
        None if shift is None else ctypes.byref(shift), ctypes.byref(out), ctypes.c_void_p(lse), ctypes.c_void_p(ws),
        ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(shape=_shape(n_layers=2)), dict(fmt=-1), dict(q=_h(31), out=_h(31)), dict(q=_h(0), out=_h(0)),
    dict(out=_h(24, 4096)), dict(dtype=3), dict(n=-1), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(scale=1e300), dict(req=_req(n_requests=-1)), dict(req=_req(max_blocks=-1)), dict(req=_req(max_queries=0)),
    dict(req=_req(table_stride=7)), dict(req=_req(block_table=None)), dict(req=_req(kv_len=None)),
    dict(req=_req(q_start=None)), dict(req=_req(kv_len=FAKE + 1)), dict(lse=FAKE + 2),
    dict(shift=H.KeyShift(FAKE, 0.0, 1)), dict(shift=H.KeyShift(FAKE, 1e4, 2)), dict(shift=H.KeyShift(None, 1e4, 1)),
    dict(q=_h(32, 4096, data=FAKE + 4)), dict(rec=_recs(block_stride_bytes=100))], ids=str)
def test_attend_refuses(kw):
    assert _attend(**kw) == H.ERR_INVALID_ARG


def test_attend_empty_and_unsupported():
    assert _attend(req=_req(n_requests=0, kv_len=None, block_table=None, q_start=FAKE)) == H.OK
    assert _attend(n=0, req=_req(q_start=FAKE)) == H.OK
    assert _attend(req=_req(n_requests=65536)) == H.ERR_UNSUPPORTED
    assert _attend(req=_req(max_blocks=1 << 28, table_stride=1 << 28)) == H.ERR_UNSUPPORTED


def test_attend_workspace_sizes():
    f = H.attend_workspace_bytes
    assert f(4, 16, 8, 4, 8, 4, 32, 1, torch.bfloat16) >= 0
    assert f(4, 16, 8, 4, 8, 4, 31, 1, torch.bfloat16) == -1          # heads not a multiple
    assert f(4, 16, 8, 4, 8, 4, 32, 0, torch.bfloat16) == -1
    assert f(4, 0, 8, 4, 8, 4, 32, 1, torch.bfloat16) == -1
    need = f(1024, 64, 8, 1, 1024, 1, 64, 1, torch.bfloat16)
    if need > 0:
        req = _req(n_requests=1, max_blocks=1024, max_queries=1, table_stride=1024)
        big = dict(shape=_shape(n_blocks=1024, block_tokens=64), rec=_recs(block_stride_bytes=133120), req=req, n=1,
                   q=_h(64, 8192), out=_h(64, 8192))
        assert _attend(**big, ws=0) == H.ERR_INVALID_ARG
        assert _attend(**big, ws=FAKE + 8) == H.ERR_INVALID_ARG
        assert _attend(**big, ws_bytes=need - 1) == H.ERR_INVALID_ARG


def test_binding_requires_gpu_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    x = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    rec = torch.zeros(4, 33280, dtype=torch.uint8)
    with pytest.raises(ValueError, match="on a GPU"):
        H.plan_step(i, i, torch.zeros(4, 8, dtype=torch.int32), i, i[:1], 16, 4)
    with pytest.raises(ValueError, match="on a GPU"):
        H.rope_heads(x, x, i, 1e4, "half_split")
    with pytest.raises(ValueError, match="on a GPU"):
        H.append_tokens(x, x, i.long(), rec, "fp8", 16)
    with pytest.raises(ValueError, match="on a GPU"):
        H.attend_records(x, rec, "fp8", 16, 8, torch.zeros(4, 8, dtype=torch.int32), i)


def test_attend_many_heads_unsupported():
    many = 4097
    shape, rec = _shape(n_kv_heads=many, block_tokens=1), _recs(block_stride_bytes=1 << 21)
    assert _attend(shape=shape, rec=rec, q=_h(many, many * 128), out=_h(many, many * 128)) == H.ERR_UNSUPPORTED
