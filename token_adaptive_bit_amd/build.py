"""Build libmbq.so (gfx950) in the package directory with hipcc, and the native binding of
the dense operators (_bind.so, host code) with the C++ compiler.  The library comes first and
needs neither Python's nor torch's headers; without those the binding is left out, and the
dense operators are called through ctypes.

Every translation unit is compiled for gfx950 only, with packed FP32 instructions
disabled (-packed-fp32-ops) and IEEE-correct float32 division.  The pack kernel is also
built with -ffp-contract=off: its float32 recursion must round every operation on its
own to reproduce the bit-exact MoBiSlice codes.

Usage:  python -m token_adaptive_bit_amd.build   (or __graft_entry__.build())
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "libmbq.so")
BIND = os.path.join(PKG, "_bind.so")
BUILD_DIR = os.path.join(ROOT, "_build")

SOURCES = {
    "api.hip": [],
    "pack.hip": ["-ffp-contract=off"],
    "route.hip": [],
    "route_mlp.hip": [],
    "lowrank.hip": [],
    "decode.hip": [],
    "decode_stream.hip": [],
    "prefill.hip": [],
    "prefill_mfma.hip": [],
    "fp8_quant.hip": [],
    "fp8_linear.hip": [],
    "block_norm.hip": [],
    "token_logprobs.hip": [],
}

# Translation units whose kernels must not spill registers: their load pipelines rely on
# exact waits on the in-order memory counter, which spill traffic (scratch loads and
# stores) would stall, and the variants a launcher can pick are chosen to fit.  The build
# reads the compiler's resource-usage remarks and fails on any spill to scratch memory.
SPILL_FREE = ("decode_stream.hip", "prefill_mfma.hip", "route_mlp.hip", "lowrank.hip",
              "fp8_quant.hip", "fp8_linear.hip", "block_norm.hip", "token_logprobs.hip")

COMMON = [
    "--offload-arch=gfx950", "-O3", "-fPIC", "-std=c++17",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-Wno-unused-result",
    "-Werror=inline-asm",  # registers that assembly may not take (m0 among its clobbers)
    "-I", os.path.join(ROOT, "include"),
]


def hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libmbq)")


def _spills(remarks: str) -> list:
    """(kernel, vgpr spills, sgpr spills, scratch bytes) of every kernel that spills to memory."""
    out, name = [], None
    vals = {}
    for line in remarks.splitlines():
        m = re.search(r"Function Name: (\S+)", line)
        if m:
            name, vals = m.group(1), {}
            continue
        for key in ("VGPRs Spill", "SGPRs Spill", "ScratchSize \\[bytes/lane\\]"):
            m = re.search(" " + key + r": (\d+)", line)
            if m:
                vals[key[:5]] = int(m.group(1))
        if name and len(vals) == 3:
            if vals["VGPRs"] or vals["Scrat"]:  # SGPR spills into VGPR lanes touch no memory
                out.append((name, vals["VGPRs"], vals["SGPRs"], vals["Scrat"]))
            name = None
    return out


def _warnings(text: str) -> list:
    """The warnings of a compiler's output; the host pass's about the GPU feature switched off in COMMON is none."""
    return [line for line in text.splitlines() if "warning:" in line and "-packed-fp32-ops" not in line]


def _compile(src: str, extra: list, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, src.replace(".hip", ".o"))
    check = src in SPILL_FREE
    remarks = ["-Rpass-analysis=kernel-resource-usage"] if check else []
    cmd = [hipcc(), *COMMON, *extra, *remarks, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{res.stdout}\n{res.stderr}")
    for line in _warnings(res.stderr):
        print(line, file=sys.stderr, flush=True)
    if check:
        bad = _spills(res.stderr)
        if bad:
            lines = "\n".join(f"  {n}: {v} VGPR / {s} SGPR spills, {b} B scratch" for n, v, s, b in bad)
            raise RuntimeError(f"{src}: kernels spill registers:\n{lines}")
    return obj


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        raise RuntimeError("torch not found (the binding is built against it)")
    return os.path.dirname(spec.origin)


def _run(cmd: list, what: str, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{res.stdout}\n{res.stderr}")


def _binding_lacks() -> str:
    """What the binding needs and this machine does not have ('' if all is there)."""
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h"
    try:
        torch = _torch_dir()
    except RuntimeError:
        return "torch"
    if not os.path.exists(os.path.join(torch, "include", "torch", "csrc", "autograd", "python_variable.h")):
        return "torch's headers"
    return ""


def _compile_bind(verbose: bool) -> str:
    """csrc/bind.cpp, the native calls of the dense operators (host code only)."""
    obj, torch = os.path.join(BUILD_DIR, "bind.o"), _torch_dir()
    cxx = shutil.which("g++") or hipcc()
    _run([cxx, "-std=c++17", "-O2", "-fPIC", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1", "-c", os.path.join(CSRC, "bind.cpp"),
          "-I", os.path.join(torch, "include"), "-I", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
          "-I", sysconfig.get_paths()["include"], "-I", "/opt/rocm/include", "-o", obj], "compiling bind.cpp", verbose)
    return obj


def _link_bind(obj: str, verbose: bool) -> None:
    lib, tmp = os.path.join(_torch_dir(), "lib"), BIND + ".tmp"
    cxx = shutil.which("g++") or hipcc()
    _run([cxx, "-shared", "-fPIC", "-o", tmp, obj, "-L", PKG, "-l:libmbq.so", "-L", lib, "-lc10", "-ltorch_cpu", "-ltorch_python",
          "-Wl,-rpath,$ORIGIN"], "linking the binding", verbose)
    os.replace(tmp, BIND)


def build(verbose: bool = False, jobs: int | None = None) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    jobs = jobs or min(len(SOURCES), max(1, min(8, os.cpu_count() or 1)))
    lacks = _binding_lacks()
    with cf.ThreadPoolExecutor(jobs) as ex:
        bind = None if lacks else ex.submit(_compile_bind, verbose)
        objs = list(ex.map(lambda kv: _compile(kv[0], kv[1], verbose), SOURCES.items()))
        tmp = OUT + ".tmp"
        _run([hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs], "link", verbose)
        os.replace(tmp, OUT)
        if bind is None:
            print(f"{os.path.basename(BIND)} not built: {lacks} not found", file=sys.stderr)
            if os.path.exists(BIND):  # of another build
                os.remove(BIND)
        else:
            _link_bind(bind.result(), verbose)
    return OUT


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
