"""What the build needs, and when a built file may be used again."""
import os
import subprocess
import sys
import sysconfig

import torch

import mamba_ssd_chunked_fwd_gb300 as ssd
from mamba_ssd_chunked_fwd_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_library_does_not_need_the_binding(monkeypatch, tmp_path):
    """The CUDA library builds and loads where the binding's headers or compiler are missing."""
    ssd.load_library()
    monkeypatch.setattr(_build, "BINDING_SRC", str(tmp_path / "missing.cpp"))

    def no_compiler(*a, **k):
        raise AssertionError("a compiler was called")
    monkeypatch.setattr(subprocess, "run", no_compiler)
    assert _build.build() == _build.LIB


def test_binding_belongs_to_its_torch_and_interpreter(monkeypatch):
    """A binding of another torch or Python is another file, so it is never imported here."""
    here = _build.build_binding()
    assert os.path.exists(here) and torch.__version__ in os.path.basename(here)
    assert sysconfig.get_config_var("SOABI") in os.path.basename(here)
    assert _build.binding_path() == here
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    assert _build.binding_path() != here


def test_binding_is_built_again_when_its_source_is_newer(monkeypatch, tmp_path):
    here = _build.build_binding()
    src = tmp_path / "binding.cpp"
    src.write_text("not C++")
    monkeypatch.setattr(_build, "BINDING_SRC", str(src))
    os.utime(src, (os.path.getmtime(here) + 10,) * 2)
    try:
        _build.build_binding()
    except RuntimeError as e:
        assert "binding" in str(e)
    else:
        raise AssertionError("the old binding was taken")
    assert os.path.exists(here)


def test_first_use_from_two_threads():
    """The binding is built and loaded once."""
    code = ("import threading, mamba_ssd_chunked_fwd_gb300 as s\n"
            "from mamba_ssd_chunked_fwd_gb300 import selective as m\n"
            "got = []\n"
            "t = [threading.Thread(target=lambda: got.append(m._binding())) for _ in range(4)]\n"
            "[i.start() for i in t]; [i.join() for i in t]\n"
            "assert len(got) == 4 and all(g is got[0] for g in got), got\n")
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True)
