"""The build's two parts: the C ABI needs nvcc alone, the torch calls follow torch."""

import subprocess
import sys

import pytest

from bit_w4a4_quantized_smooth_b200 import binding, build


@pytest.fixture(autouse=True)
def built():
    build.build()


def test_c_abi_builds_without_torch(tmp_path):
    """With torch not importable the build still gives libsvdq.so and says what it left out."""
    code = ("import sys; sys.modules['torch'] = None\n"
            "import os; sys.path.insert(0, os.getcwd())\n"
            "from bit_w4a4_quantized_smooth_b200 import build\n"
            "print(build.build())\n")
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.strip() == build.LIB and "torch cannot be imported" in r.stderr


@pytest.mark.parametrize("what", ["Python.h", "g++"])
def test_c_abi_builds_without_headers_or_compiler(monkeypatch, capsys, what):
    if what == "g++":
        monkeypatch.setattr(build.shutil, "which", lambda name: None)
    else:
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": "/nonexistent"})
    monkeypatch.setattr(build, "build_torch_calls", lambda: pytest.fail("tried to build the torch calls"))
    monkeypatch.setattr(build, "TORCH_LIB", "/nonexistent/_svdq_torch.so")
    assert build.build() == build.LIB
    assert what in capsys.readouterr().err


def test_torch_calls_are_built_again_for_another_torch(monkeypatch):
    calls = []
    monkeypatch.setattr(build, "build_torch_calls", lambda: calls.append(1))
    build.build()
    assert not calls
    monkeypatch.setattr(build, "torch_tag", lambda: "torch 0.0.1, cpython-312")
    build.build()
    assert calls


def test_torch_calls_of_another_torch_are_refused(monkeypatch):
    monkeypatch.setattr(binding, "_ext", None)
    assert binding._native().built_for == build.torch_tag()
    monkeypatch.setattr(binding, "_ext", None)
    monkeypatch.setattr(build, "torch_tag", lambda: "torch 0.0.1, cpython-312")
    with pytest.raises(ImportError, match="0.0.1"):
        binding._native()
