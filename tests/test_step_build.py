"""What a build of the C library asks for: hipcc alone; the Python module beside it needs torch's
headers and is left out where there are none."""

import os
import subprocess
import sys
import types

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_build_without_torch_leaves_out_the_python_module(tmp_path):
    code = ("import sys; sys.modules['torch'] = None\n"
            "from gemv_prefill_decode_amd import build as b\n"
            f"b.STEP_OUT = {str(tmp_path / '_step.so')!r}\n"
            "assert b.build_step() == ''\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "_step.so is not built" in r.stderr and not os.listdir(tmp_path)


def test_python_module_is_compiled_by_the_same_compiler(monkeypatch, tmp_path):
    from gemv_prefill_decode_amd import build as b
    try:
        compiler = b.hipcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    used = []

    def run(cmd, **kw):
        used.append(cmd[0])
        return types.SimpleNamespace(returncode=1, stdout="", stderr="stopped")

    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.setattr(b, "STEP_OUT", str(tmp_path / "_step.so"))
    with pytest.raises(RuntimeError, match="stopped"):
        b.build_step()
    assert used == [compiler]
