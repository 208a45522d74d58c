"""The page serving calls' argument checks, on the host: bad arguments are
refused before any HIP call (no GPU needed), empty calls launch nothing, the
header is plain C99 and every function it declares is exported."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from quantization_rope_reuse_amd import hkv as H

FAKE = 0x7F0000000000          # a 16-byte aligned address never dereferenced
HEADER = os.path.join(os.path.dirname(H.HEADER), "hkv_pages.h")


def declared():
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return sorted(set(re.findall(r"\b(hkv_[a-z0-9_]+)\s*\(", text)))


def test_exports_every_declared_symbol():
    assert declared() == ["hkv_append_pages", "hkv_attend_pages", "hkv_attend_pages_workspace_bytes",
                          "hkv_join_attention"]
    for n in declared():
        assert getattr(H.lib(), n) is not None


def test_header_is_plain_c_and_sizes_match(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("needs gcc and the ROCm headers")
    src = tmp_path / "uses.c"
    src.write_text('#include <stdio.h>\n#include "hkv_pages.h"\nint main(void) {\n'
                   + "".join(f"  (void)&{n};\n" for n in declared())
                   + '  printf("%zu\\n", sizeof(hkv_scores));\n'
                   "  return hkv_join_attention(0, 0, 0, 0, 0, 0, 0, 0, 0) == HKV_ERR_INVALID_ARG ? 0 : 1;\n}\n")
    pkg = os.path.dirname(H.LIB_PATH)
    exe = tmp_path / "uses"
    r = subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__",
                        "-I", "/opt/rocm/include", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe),
                        "-L", pkg, "-lhkv", f"-Wl,-rpath,{pkg}"], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and int(r.stdout) == ctypes.sizeof(H.Scores)


def _h(heads=8, tok=1024, head=128, data=FAKE):
    return H.Heads(data, tok, head, heads)


def _shape(**kw):
    d = dict(n_layers=1, n_blocks=4, block_tokens=16, n_kv_heads=8, head_dim=128)
    d.update(kw)
    return H.Shape(**d)


def _pages(**kw):
    d = dict(k=FAKE, v=FAKE + (1 << 30), layer_stride=0, page_stride=16 * 1024, token_stride=1024, head_stride=128,
             num_pages=4)
    d.update(kw)
    return H.Pages(**d)


def _ref(x):
    return None if x is None else ctypes.byref(x)


# --- append ----------------------------------------------------------------

def _append(shape=None, axes=None, rope=True, pos=FAKE, axis_stride=32, q=None, k=None, v=None, qo=None, dtype=2, n=32,
            slots=FAKE, pages=None, page_dtype=2):
    a = H.rope_axes(1e4, "half_split", (16, 24, 24)) if axes is None else axes
    q, qo = (x if x is not None else _h(32, 4096) for x in (q, qo))
    k, v = (x if x is not None else _h() for x in (k, v))
    shape, pages = shape or _shape(), pages or _pages()
    return H.lib().hkv_append_pages(_ref(shape), _ref(a) if rope else None, ctypes.c_void_p(pos), axis_stride, _ref(q),
                                    _ref(k), _ref(v), _ref(qo), dtype, n, ctypes.c_void_p(slots), _ref(pages),
                                    page_dtype, None)


@pytest.mark.parametrize("kw", [
    dict(shape=_shape(n_layers=2)), dict(shape=_shape(n_blocks=5)), dict(shape=_shape(head_dim=64)),
    dict(shape=_shape(block_tokens=0)), dict(pages=_pages(num_pages=3)), dict(pages=_pages(k=0)),
    dict(pages=_pages(v=FAKE + 8)), dict(pages=_pages(token_stride=4)), dict(pages=_pages(page_stride=-1024)),
    dict(pages=_pages(page_stride=1 << 46)), dict(axes=H.RopeAxes(0, 1, 1e4)), dict(axes=H.RopeAxes(1, 2, 1e4)),
    dict(axes=H.RopeAxes(1, 1, 0.0)), dict(pos=0), dict(pos=FAKE + 2), dict(axis_stride=-1), dict(n=-1), dict(dtype=3),
    dict(page_dtype=-1), dict(slots=0), dict(slots=FAKE + 4), dict(k=_h(7)), dict(v=_h(9)), dict(qo=_h(31, 4096)),
    dict(q=_h(32, 4096, data=FAKE + 8)), dict(k=_h(data=0)), dict(v=_h(tok=4)), dict(rope=False)], ids=str)
def test_append_refuses(kw):
    assert _append(**kw) == H.ERR_INVALID_ARG


def test_append_empty_and_unsupported():
    assert _append(n=0, pos=0, slots=0) == H.OK
    none = _h(0, 0, 0, 0)
    assert _append(rope=False, pos=0, q=none, qo=none, n=0) == H.OK
    many = _h(1 << 24, 0, 0)
    assert _append(q=many, qo=many) == H.ERR_UNSUPPORTED
    assert _append(n=1 << 27, axis_stride=1 << 27) == H.ERR_UNSUPPORTED


# --- attend ----------------------------------------------------------------

def _req(**kw):
    d = dict(n_requests=4, max_blocks=8, max_queries=1, block_table=FAKE, table_stride=8, kv_len=FAKE, q_start=FAKE)
    d.update(kw)
    return H.Requests(**d)


def _scores(**kw):
    d = dict(sm_scale=0.1, cap=0.0, causal=1, window=0, positions=None, begin=None, prefix_len=None, slopes=None)
    d.update(kw)
    return H.Scores(**d)


def _attend(shape=None, pages=None, req=None, q=None, dtype=2, n=4, scores=None, out=None, lse=FAKE, ws=FAKE,
            ws_bytes=1 << 30, no_scores=False):
    q, out = (x if x is not None else _h(32, 4096) for x in (q, out))
    shape, pages, req, scores = shape or _shape(), pages or _pages(), req or _req(), scores or _scores()
    return H.lib().hkv_attend_pages(_ref(shape), _ref(pages), _ref(req), _ref(q), dtype, n,
                                    None if no_scores else _ref(scores), _ref(out), ctypes.c_void_p(lse),
                                    ctypes.c_void_p(ws), ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(shape=_shape(n_layers=2)), dict(shape=_shape(n_blocks=3)), dict(pages=_pages(k=0)), dict(pages=_pages(num_pages=9)),
    dict(pages=_pages(head_stride=-128)), dict(pages=_pages(head_stride=4)), dict(q=_h(31), out=_h(31)),
    dict(q=_h(0), out=_h(0)), dict(out=_h(24, 4096)), dict(dtype=3), dict(n=-1), dict(no_scores=True),
    dict(scores=_scores(sm_scale=float("nan"))), dict(scores=_scores(sm_scale=float("inf"))),
    dict(scores=_scores(cap=-1.0)), dict(scores=_scores(cap=float("nan"))), dict(scores=_scores(cap=float("inf"))),
    dict(scores=_scores(window=-1)), dict(scores=_scores(positions=FAKE + 2)), dict(scores=_scores(begin=FAKE + 1)),
    dict(scores=_scores(prefix_len=FAKE + 3)), dict(scores=_scores(slopes=FAKE + 2)), dict(req=_req(n_requests=-1)),
    dict(req=_req(max_blocks=-1)), dict(req=_req(max_queries=0)), dict(req=_req(table_stride=7)),
    dict(req=_req(block_table=None)), dict(req=_req(kv_len=None)), dict(n=5, req=_req(q_start=None)),
    dict(req=_req(kv_len=FAKE + 1)), dict(lse=FAKE + 2), dict(q=_h(32, 4096, data=FAKE + 4))], ids=str)
def test_attend_refuses(kw):
    assert _attend(**kw) == H.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(scores=_scores(sm_scale=1e31)), dict(scores=_scores(sm_scale=-1e31)), dict(scores=_scores(cap=1e31)),
    dict(scores=_scores(cap=1e-31)), dict(scores=_scores(cap=1e-20, sm_scale=1e20)), dict(req=_req(n_requests=65536)),
    dict(req=_req(max_blocks=1 << 28, table_stride=1 << 28)), dict(n=1 << 27),
    dict(shape=_shape(n_kv_heads=4097, block_tokens=1), q=_h(4097, 4097 * 128), out=_h(4097, 4097 * 128))], ids=str)
def test_attend_unsupported(kw):
    assert _attend(**kw) == H.ERR_UNSUPPORTED


def test_attend_empty():
    assert _attend(req=_req(n_requests=0, kv_len=None, block_table=None)) == H.OK
    assert _attend(n=0) == H.OK


def test_attend_workspace_sizes():
    f = H.attend_pages_workspace_bytes
    assert f(4, 16, 8, 4, 8, 4, 32, 1, torch.bfloat16) >= 0
    assert f(4, 16, 8, 4, 8, 4, 31, 1, torch.bfloat16) == -1          # heads not a multiple
    assert f(4, 16, 8, 4, 8, 4, 32, 0, torch.bfloat16) == -1
    assert f(4, 0, 8, 4, 8, 4, 32, 1, torch.bfloat16) == -1
    need = f(1024, 64, 8, 1, 1024, 1, 64, 1, torch.bfloat16)
    assert need > 0
    big = dict(shape=_shape(n_blocks=1024, block_tokens=64), pages=_pages(num_pages=1024, page_stride=64 * 1024),
               req=_req(n_requests=1, max_blocks=1024, table_stride=1024), n=1, q=_h(64, 8192), out=_h(64, 8192))
    assert _attend(**big, ws=0) == H.ERR_INVALID_ARG
    assert _attend(**big, ws=FAKE + 8) == H.ERR_INVALID_ARG
    assert _attend(**big, ws_bytes=need - 1) == H.ERR_INVALID_ARG


# --- join ------------------------------------------------------------------

def _join(a=None, b=None, o=None, la=FAKE, lb=FAKE, lo=FAKE, dtype=2, n=4):
    a, b, o = (x if x is not None else _h() for x in (a, b, o))
    return H.lib().hkv_join_attention(_ref(a), ctypes.c_void_p(la), _ref(b), ctypes.c_void_p(lb), dtype, n, _ref(o),
                                      ctypes.c_void_p(lo), None)


@pytest.mark.parametrize("kw", [dict(a=_h(7)), dict(b=_h(9)), dict(o=_h(4)), dict(la=0), dict(lb=0), dict(la=FAKE + 2),
                                dict(lo=FAKE + 1), dict(dtype=5), dict(n=-1), dict(a=_h(data=FAKE + 8)), dict(b=_h(data=0)),
                                dict(o=_h(tok=4)), dict(o=_h(head=-128)), dict(a=_h(tok=1 << 47))], ids=str)
def test_join_refuses(kw):
    assert _join(**kw) == H.ERR_INVALID_ARG


def test_join_empty_and_unsupported():
    assert _join(n=0, la=0, lb=0) == H.OK
    none = _h(0, 0, 0, 0)
    assert _join(a=none, b=none, o=none, la=0, lb=0, lo=0) == H.OK
    assert _join(n=1 << 29) == H.ERR_UNSUPPORTED


def test_binding_requires_gpu_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    x = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    p = torch.zeros(4, 16, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="on a GPU"):
        H.append_pages(x, x, i.long(), p, p)
    with pytest.raises(ValueError, match="on a GPU"):
        H.attend_pages(x, p, p, torch.zeros(4, 8, dtype=torch.int32), i)
    with pytest.raises(ValueError, match="on a GPU"):
        H.join_attention(x, x[..., 0].float(), x, x[..., 0].float())
