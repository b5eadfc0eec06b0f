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
    "int8_quant.hip": [],
    "int8_linear.hip": [],
    "experts.hip": [],
}

# Translation units whose kernels must not spill registers: their load pipelines rely on
# exact waits on the in-order memory counter, which spill traffic (scratch loads and
# stores) would stall, and the variants a launcher can pick are chosen to fit.  The build
# reads the compiler's resource-usage remarks and fails on any spill to scratch memory.
SPILL_FREE = ("decode_stream.hip", "prefill_mfma.hip", "route_mlp.hip", "lowrank.hip",
              "fp8_quant.hip", "fp8_linear.hip", "block_norm.hip", "token_logprobs.hip",
              "int8_quant.hip", "int8_linear.hip", "experts.hip")

# Translation units whose assembly is read: waits that count the compiler's own loads.
COUNTED_WAITS = ("int8_linear.hip",)

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


_WAIT = re.compile(r"s_waitcnt vmcnt\((\d+)\) ; at most (\d+) copies of the youngest")
_VMEM = re.compile(r"(global|buffer|flat|scratch)_(load|store|atomic)")
_COPY = re.compile(r"(global|buffer)_load_lds|buffer_load\w* .*\blds\b")


def _late_copies(assembly: str) -> list:
    """What is wrong with the counted waits of an assembly: (kernel, line, N, copies allowed, copies found) where on some way to
    a wait more of the N youngest vector memory operations are copies than it says; (kernel, 0, 0, 0, 0) for no wait at all."""
    bad, name, waits = [], None, 0
    ops, labels = [], {}                   # ops: (kind, what, line number); kind of "op", "copy", "wait", "end", "go", "maybe", "-"

    def check():
        back = [[] for _ in ops]           # where each operation can be reached from
        for i, (kind, what, _) in enumerate(ops):
            if i + 1 < len(ops) and kind not in ("end", "go"):
                back[i + 1].append(i)
            if kind in ("go", "maybe") and labels.get(what, len(ops)) < len(ops):
                back[labels[what]].append(i)
        for i, (kind, what, line) in enumerate(ops):
            if kind != "wait":
                continue
            n, allowed = what
            worst, seen, todo = 0, set(), [(j, n, 0) for j in back[i]]
            while todo:
                at, left, copies = state = todo.pop()
                if state in seen or left == 0:
                    continue
                seen.add(state)
                if ops[at][0] in ("op", "copy"):
                    left, copies = left - 1, copies + (ops[at][0] == "copy")
                    worst = max(worst, copies)
                todo += [(j, left, copies) for j in back[at]]
            if worst > allowed:
                bad.append((name, line, n, allowed, worst))

    for number, text in enumerate(assembly.splitlines(), 1):
        word = text.strip()
        if re.match(r"_Z\w+:", word):
            name, ops, labels, waits = word.split(":")[0], [], {}, 0
        elif name is None or not word:
            continue
        elif word.startswith(".Lfunc_end"):
            check()
            if "direct_kernel" in name and not waits:
                bad.append((name, 0, 0, 0, 0))
            name = None
        elif re.match(r"\.L\w+:", word):
            labels[word.split(":")[0]] = len(ops)
            ops.append(("-", None, number))
        elif _WAIT.search(word):
            ops.append(("wait", tuple(map(int, _WAIT.search(word).groups())), number))
            waits += 1
        elif word.startswith((";", ".")):
            continue
        elif _COPY.match(word):
            ops.append(("copy", None, number))
        elif _VMEM.match(word):
            ops.append(("op", None, number))
        elif word.startswith("s_endpgm"):
            ops.append(("end", None, number))
        elif word.startswith("s_branch"):
            ops.append(("go", word.split()[1], number))
        elif word.startswith("s_cbranch"):
            ops.append(("maybe", word.split()[1], number))
        elif word.startswith(("s_setpc", "s_swappc", "s_call")):
            bad.append((name, number, 0, 0, 0))
    return bad


def _assembly(src: str, extra: list) -> str:
    """The GPU assembly of a translation unit."""
    out = os.path.join(BUILD_DIR, src.replace(".hip", ".s"))
    _run([hipcc(), *COMMON, *extra, "--cuda-device-only", "-S", os.path.join(CSRC, src), "-o", out], f"compiling {src} to assembly", False)
    with open(out) as f:
        return f.read()


def _check_waits(src: str, extra: list) -> None:
    bad = _late_copies(_assembly(src, extra))
    if bad:
        lines = "\n".join(f"  {k}, line {line}: of the {n} youngest operations {found} may be copies, {allowed} are allowed"
                          for k, line, n, allowed, found in bad)
        raise RuntimeError(f"{src}: waits that may pass before a copy is in:\n{lines}")


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
    if src in COUNTED_WAITS:
        _check_waits(src, extra)
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
