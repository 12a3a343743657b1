"""The C library builds where PyTorch is not there (no GPU)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _run(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


def test_c_library_builds_without_torch():
    r = _run("import sys; sys.modules['torch'] = None\n"
             "from swiglu_gemm_transformer_gb300 import _build\n"
             "import swiglu_gemm_transformer_gb300 as sg\n"
             "assert _build.build() == sg.LIB_PATH\n"
             "assert sg.lib().swiglu_moe_route_workspace_size(1, 64, 8) == 0\n")
    assert r.returncode == 0, r.stderr
    assert "_swiglu_torch" in r.stderr      # says what was left out


def test_c_library_builds_with_a_torch_without_cuda(monkeypatch, capsys):
    import torch

    from swiglu_gemm_transformer_gb300 import _build
    monkeypatch.setattr(torch.version, "cuda", None)
    assert _build.build() == _build.LIB
    assert "_swiglu_torch" in capsys.readouterr().err


def test_calls_of_the_torch_module_say_that_it_is_missing(monkeypatch, tmp_path):
    import torch

    import swiglu_gemm_transformer_gb300 as sg
    monkeypatch.setattr(sg, "_torch_mod", None)
    monkeypatch.setattr(sg, "TORCH_LIB_PATH", str(tmp_path / "none.so"))
    with pytest.raises(RuntimeError, match="PyTorch"):
        sg.swiglu_moe_route(torch.zeros(2, 4), 1)
