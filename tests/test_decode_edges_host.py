"""What the plain-decoding and 8-bit-cache calls rest on, as far as it shows without a GPU."""

import importlib
import os
import re
import subprocess
import sys

import pytest
import torch

import speculative_decoding_tree_build_gb300 as tv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "speculative_decoding_tree_build_gb300")
CSRC = os.path.join(PKG, "csrc")


def test_no_launch_rule_holds_a_number_of_sms():
    """Launch rules ask the device (device_sm_count) and do not reckon with one GPU's 152 SMs."""
    for f in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, f), encoding="utf-8") as fh:
            code = re.sub(r"//[^\n]*|/\*.*?\*/", "", fh.read(), flags=re.S)
        assert not re.findall(r"\b152\s*\*|[*/]\s*\(?\s*152\b", code), f


def test_the_library_is_built_though_the_binding_does_not_compile(tmp_path, monkeypatch):
    made = small_build(monkeypatch, tmp_path)

    def fails(nvcc):
        raise RuntimeError("the binding does not compile")

    monkeypatch.setattr(made, "_compile_binding", fails)
    with pytest.raises(RuntimeError, match="binding does not compile"):
        made.build()
    assert os.path.exists(made.LIB) and not os.path.exists(made.EXT)
    # it is asked for again, and the library is not compiled again for it
    seen = os.stat(made.LIB).st_mtime_ns
    with pytest.raises(RuntimeError, match="binding does not compile"):
        made.build()
    assert made.build(bindings=False) == made.LIB and os.stat(made.LIB).st_mtime_ns == seen


def small_build(monkeypatch, where):
    """The package's build in a directory of its own, of one translation unit."""
    made = importlib.import_module("speculative_decoding_tree_build_gb300.build")
    monkeypatch.setattr(made, "BUILD", str(where / "build"))
    monkeypatch.setattr(made, "LIB", str(where / "lib.so"))
    monkeypatch.setattr(made, "EXT", str(where / "ext.so"))
    monkeypatch.setattr(made, "_sources", lambda: [os.path.join(CSRC, "api.cu")])
    return made


def test_the_library_is_built_without_torch(tmp_path):
    code = f"""
import importlib.util, os, sys
sys.modules["torch"] = None                       # import torch fails
spec = importlib.util.spec_from_file_location("lone_build", {os.path.join(PKG, 'build.py')!r})
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
b.BUILD, b.LIB, b.EXT = {str(tmp_path / 'build')!r}, {str(tmp_path / 'lib.so')!r}, {str(tmp_path / 'ext.so')!r}
b._sources = lambda: [os.path.join(b.CSRC, "api.cu")]
print(b.build(bindings=False))
"""
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    assert os.path.exists(tmp_path / "lib.so") and not os.path.exists(tmp_path / "ext.so")


def test_an_extension_built_for_another_torch_is_refused(monkeypatch):
    importlib.import_module("speculative_decoding_tree_build_gb300.build").build()
    monkeypatch.setattr(tv, "_ext", None)
    assert tv._native().torch_version == torch.__version__
    monkeypatch.setattr(tv, "_ext", None)
    monkeypatch.setattr(torch, "__version__", "0.1.0")
    with pytest.raises(ImportError, match="built for torch"):
        tv._native()
