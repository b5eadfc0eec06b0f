"""What the build does with the compiler's warnings (no GPU)."""
import subprocess

import pytest

from token_adaptive_bit_amd import build as B


def test_warnings_of_a_successful_compile_are_shown(monkeypatch, tmp_path, capsys):
    text = "'-packed-fp32-ops' is not a recognized feature for this target (ignoring feature)\na.hip:3:1: warning: something\n"
    monkeypatch.setattr(B, "hipcc", lambda: "hipcc")
    monkeypatch.setattr(B, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(B.subprocess, "run", lambda cmd, **kw: subprocess.CompletedProcess(cmd, 0, "", text))
    B._compile("api.hip", [], False)
    err = capsys.readouterr().err
    assert "a.hip:3:1: warning: something" in err and "recognized" not in err


@pytest.mark.parametrize("clobbers,ok", [('"memory"', True), ('"memory", "m0"', False)])
def test_assembly_may_not_take_reserved_registers(tmp_path, clobbers, ok):
    try:
        hipcc = B.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    src = tmp_path / "a.hip"
    src.write_text('#include <hip/hip_runtime.h>\n__global__ void f() { asm volatile("s_nop 0" ::: ' + clobbers + "); }\n")
    res = subprocess.run([hipcc, *B.COMMON, "-c", str(src), "-o", str(tmp_path / "a.o")], capture_output=True, text=True)
    assert (res.returncode == 0) is ok, res.stderr
