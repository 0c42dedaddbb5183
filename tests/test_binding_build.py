"""The native part of the binding: built beside the library, and not needed for it."""
import os
import subprocess
import sys

import pytest

from kda_delta_rule_gb300 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


def test_native_binding_is_there():
    B.build()
    r = _python("from kda_delta_rule_gb300 import kda\n"
                "assert kda._native.__file__.endswith('_kda_torch.so')")
    assert r.returncode == 0, r.stderr


def test_import_without_the_native_binding():
    """Every entry point is there, with a warning; refusals come from the way through ctypes."""
    B.build()
    r = _python("import sys, warnings\n"
                "sys.modules['kda_delta_rule_gb300._kda_torch'] = None\n"
                "with warnings.catch_warnings(record=True) as w:\n"
                "    warnings.simplefilter('always')\n"
                "    from kda_delta_rule_gb300 import kda\n"
                "assert any('ctypes' in str(x.message) for x in w)\n"
                "import torch\n"
                "assert kda._native is None and kda.kda_mla_decode_workspace_bytes(1, 1, 32, 512, 0, torch.bfloat16) > 0\n"
                "try:\n"
                "    kda.kda_mla_decode(torch.zeros(1, 1, 1, 128), None, None, 16, None, None, 1.0)\n"
                "except TypeError as e:\n"
                "    print('refused:', e)\n")
    assert r.returncode == 0 and "refused: q must be a CUDA tensor" in r.stdout, r.stderr


def _elsewhere(monkeypatch, tmp_path):
    """The build's outputs in a folder of their own, the library taken as built."""
    for name in ("LIB", "BINDING_LIB", "BINDING_FOR"):
        monkeypatch.setattr(B, name, str(tmp_path / os.path.basename(getattr(B, name))))
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "_build"))
    (tmp_path / "libkda.so").touch()


def test_build_goes_on_without_the_native_binding(monkeypatch, tmp_path):
    """No host compiler for it: the library is built all the same, an older binding does not stay beside it."""
    _elsewhere(monkeypatch, tmp_path)
    (tmp_path / "_kda_torch.so").touch()
    os.utime(tmp_path / "_kda_torch.so", (1, 1))

    def none():
        raise RuntimeError("no C++ compiler found for the Python binding")

    monkeypatch.setattr(B, "_cxx", none)
    with pytest.warns(RuntimeWarning, match="ctypes"):
        assert B.build() == str(tmp_path / "libkda.so")
    assert not (tmp_path / "_kda_torch.so").exists()


def test_native_binding_is_rebuilt_for_another_pytorch(monkeypatch, tmp_path):
    """Newer than every source, but made for another PyTorch."""
    _elsewhere(monkeypatch, tmp_path)
    made = []
    monkeypatch.setattr(B, "_build_binding", lambda nvcc: ("binding.o", "torch/lib"))
    monkeypatch.setattr(B, "_run", lambda cmd, what: (made.append(what), open(cmd[cmd.index("-o") + 1], "w").close()))
    B.build()
    assert made == ["the binding's link"] and B.binding_made_for() == B.this_torch()
    B.build()
    assert len(made) == 1
    monkeypatch.setattr(B, "this_torch", lambda: "torch 0.0, another Python")
    B.build()
    assert len(made) == 2


def test_import_of_a_native_binding_for_another_pytorch():
    """It is not loaded: its idea of a tensor may differ where the symbols do not."""
    B.build()
    r = _python("from kda_delta_rule_gb300 import build\n"
                "build.this_torch = lambda: 'torch 0.0, another Python'\n"
                "import warnings\n"
                "with warnings.catch_warnings(record=True) as w:\n"
                "    warnings.simplefilter('always')\n"
                "    from kda_delta_rule_gb300 import kda\n"
                "assert kda._native is None and any('this is torch 0.0' in str(x.message) for x in w)\n")
    assert r.returncode == 0, r.stderr
