"""Build libhkv.so (HIP, gfx950) and the native part of the binding in place,
next to this file.

    python -m quantization_rope_reuse_amd.build

Each source is compiled to an object under _build/ in parallel, then linked
into one shared library.  Flags: -O3 without any fast-math option, so fp32
division and square root stay correctly rounded and denormals are kept; the
packed-fp32 feature is disabled for the device code.
"""

from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libhkv.so")
SOURCES = ("api.hip", "quant.hip", "fetch.hip", "crc.hip", "order.hip", "streams.hip",
           "select.hip", "frames.hip", "probe.hip", "noalloc.hip",
           "staged.hip", "serve_api.hip", "plan.hip", "rope.hip", "append.hip", "attend.hip",
           "attend_rows_int4.hip", "attend_rows_fp8.hip",
           "attend_prompt_int4.hip", "attend_prompt_fp8.hip", "pages_api.hip", "append_pages.hip",
           "join.hip", "attend_pages.hip",
           *(f"attend_pages_{kind}_{t}.hip" for kind in ("rows", "chunk")
             for t in ("bf16", "f16", "f32")))
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (set HIPCC or install ROCm)")


def compile_flags():
    return [
        f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
        "-Wall", "-Wno-unused-function",
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-I", INCLUDE, "-I", CSRC,
    ]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(l for l in r.stdout.splitlines()
                    if "packed-fp32-ops' is not a recognized feature" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"command failed ({r.returncode}): {' '.join(cmd)}\n{out}")
    if verbose and out.strip():
        print(out, flush=True)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = hipcc()
    objs = []
    jobs = []
    for src in SOURCES:
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        objs.append(obj)
        jobs.append([cc, *compile_flags(), "-c", os.path.join(CSRC, src), "-o", obj])
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(jobs))) as ex:
        for f in [*(ex.submit(_run, j, verbose) for j in jobs), ex.submit(build_native, verbose)]:
            f.result()
    tmp = LIB + ".tmp"
    _run([cc, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs], verbose)
    os.replace(tmp, LIB)
    return LIB


def build_native(verbose: bool = False) -> str:
    """The native part of the Python binding (host code only)."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import TORCH_LIB_PATH, include_paths
    out = os.path.join(PKG, "_native.so")
    tmp = out + ".tmp"
    flags = [f"-I{d}" for d in (*include_paths(), "/opt/rocm/include", INCLUDE,
                                sysconfig.get_paths()["include"])]
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__",
          "-DUSE_ROCM", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *flags,
          os.path.join(CSRC, "binding.cpp"), "-o", tmp, f"-L{TORCH_LIB_PATH}", "-ltorch_python",
          "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_hip"], verbose)
    os.replace(tmp, out)
    return out


def build_test_kernels(verbose: bool = False) -> list:
    """Test-only HIP libraries under tests/hip/ (each built from one source
    with the library's flags and device headers); the GPU tests load them."""
    cc = hipcc()
    out = []
    tests_hip = os.path.join(ROOT, "tests", "hip")
    for src in sorted(os.listdir(tests_hip)):
        if not src.endswith(".hip"):
            continue
        lib = os.path.join(tests_hip, "lib" + os.path.splitext(src)[0] + ".so")
        _run([cc, *compile_flags(), "-shared", os.path.join(tests_hip, src), "-o", lib + ".tmp"],
             verbose)
        os.replace(lib + ".tmp", lib)
        out.append(lib)
    return out


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
