"""The package without its native binding (no GPU): the library and the routed operators need
only libmbq.so, and the dense operators then go through ctypes."""
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = """
import sys, warnings
sys.modules["token_adaptive_bit_amd._bind"] = None        # as if it were not there
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    from token_adaptive_bit_amd import api
assert any("native binding" in str(w.message) for w in seen)
assert api.describe(64, 256, 64, 3).n == 64
sys.path.insert(0, "tests")
import test_dense_validation as V
r = V.Recorder(V.L)
V._lib.LIB, api._stream_of = r, lambda x: None
V.test_binding_forwards(r)
"""


def test_api_without_the_binding():
    res = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-3000:]


@pytest.mark.parametrize("lacks", ["", "torch's headers"])
def test_the_library_is_built_without_the_binding(monkeypatch, tmp_path, lacks):
    """Where the binding cannot be built or fails to, the library is in place."""
    from token_adaptive_bit_amd import build as B
    out, bind = tmp_path / "libmbq.so", tmp_path / "_bind.so"
    bind.write_text("of another build")

    def run(cmd, what, verbose):
        if what != "link":
            raise RuntimeError(what)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(B, "OUT", str(out))
    monkeypatch.setattr(B, "BIND", str(bind))
    monkeypatch.setattr(B, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(B, "hipcc", lambda: "hipcc")
    monkeypatch.setattr(B, "_compile", lambda src, extra, verbose: src)
    monkeypatch.setattr(B, "_run", run)
    monkeypatch.setattr(B, "_binding_lacks", lambda: lacks)
    if lacks:
        B.build()
        assert not bind.exists()
    else:
        with pytest.raises(RuntimeError):
            B.build()                                          # the binding's own error
    assert out.exists()
