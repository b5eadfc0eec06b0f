"""The integer and expert operators' host code (validation, plans and workspace sizes) under the address
and undefined-behaviour sanitizers: api.hip and the operators' files compiled with them on
the host side only, and tests/expert_host_check.cpp, run with no GPU visible."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OUT = os.path.join(ROOT, "_build", "asan_expert")
FILES = ("api.hip", "int8_quant.hip", "int8_linear.hip", "experts.hip")


def test_expert_host_code_is_sanitizer_clean():
    from token_adaptive_bit_amd import build as B
    try:
        hipcc = B.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    rest = [os.path.join(B.BUILD_DIR, s.replace(".hip", ".o")) for s in B.SOURCES if s not in FILES]
    if not all(os.path.exists(o) for o in rest):
        B.build()
    os.makedirs(OUT, exist_ok=True)
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    objs, exe, drv = [], os.path.join(OUT, "expert_host_check"), os.path.join(OUT, "expert_host_check.o")
    steps = []
    for f in FILES:
        objs.append(os.path.join(OUT, f.replace(".hip", ".o")))
        steps.append([hipcc, *B.COMMON, "-g", *san, "-c", os.path.join(B.CSRC, f), "-o", objs[-1]])
    steps += [["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
               "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", "/opt/rocm/include",
               "-c", os.path.join(ROOT, "tests", "expert_host_check.cpp"), "-o", drv],
              [hipcc, "--offload-arch=gfx950", *san, drv, *objs, *rest, "-o", exe]]
    for cmd in steps:
        res = subprocess.run(cmd, capture_output=True, text=True)
        assert res.returncode == 0, res.stderr[-4000:]
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", ASAN_OPTIONS="detect_leaks=0:verify_asan_link_order=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1")
    env.pop("LD_PRELOAD", None)
    res = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-2000:]
