"""The library and the compiled bindings are built apart: the W8A8 calls need no headers of Python
or torch, and bindings made for another Python or torch are made again."""
import os
import shutil
import subprocess
import sys

import pytest

import w8a8_quantized_projections_gb300 as clef
from w8a8_quantized_projections_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_library_loads_without_the_extension():
    """In a process of its own: no extension is there, and compiling one fails."""
    clef.library()
    code = ("import w8a8_quantized_projections_gb300 as clef\n"
            "from w8a8_quantized_projections_gb300 import build\n"
            "def fail(*a):\n    raise RuntimeError('no Python.h')\n"
            "build.EXT, build.KEY = build.EXT + '.none', build.KEY + '.none'\n"
            "build._compile_extension = fail\n"
            "assert clef.library().clef_abi_version() == 100\n"
            "try:\n    clef.w4_linear(None, None, None)\n"
            "except RuntimeError as e:\n    assert 'no Python.h' in str(e)\n"
            "else:\n    raise AssertionError('the bindings are there')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.fixture
def built(tmp_path, monkeypatch):
    build.build()
    for name in ("EXT", "KEY"):
        shutil.copy2(getattr(build, name), tmp_path)
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    made = []
    monkeypatch.setattr(build, "_compile_extension", lambda: made.append("compiled") or "py_decode.o")
    monkeypatch.setattr(build, "_link_extension", lambda obj: made.append("linked"))
    return made


def test_extension_is_kept(built):
    assert build.build_extension() == build.EXT and not built


@pytest.mark.parametrize("change", ["torch", "python", "no key", "no extension"])
def test_extension_is_made_again(built, monkeypatch, change):
    if change == "torch":
        other = os.path.join(os.path.dirname(build.EXT), "torch")
        os.mkdir(other)
        with open(os.path.join(other, "version.py"), "w") as f:
            f.write("__version__ = '0.0'\n")
        monkeypatch.setattr(build, "_torch_dir", lambda: other)
    elif change == "python":
        monkeypatch.setattr(build.sys, "version", "0.0")
    else:
        os.remove(build.KEY if change == "no key" else build.EXT)
    build.build_extension()
    assert built == ["compiled", "linked"]
