"""The build's choices, with no compiler run: what is built without torch, and when the
module that uses torch is built again."""
import importlib.util
import os
import subprocess
import sys

import pytest

from lossless_bit_weight_encode_gb300 import build as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class FakeCompiler:
    """Stands for subprocess.Popen and run: every command leaves its output file."""

    def __init__(self):
        self.commands = []

    def __call__(self, cmd, **kw):
        self.commands.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        self.returncode = 0
        self.stdout = ""
        return self

    def communicate(self):
        return "", None

    def outputs(self):
        return [os.path.basename(c[c.index("-o") + 1]).split(".tmp")[0] for c in self.commands]


@pytest.fixture
def fake(tmp_path, monkeypatch):
    for name in ("LIB_PATH", "KV_HOST_PATH"):
        monkeypatch.setattr(b, name, str(tmp_path / os.path.basename(getattr(b, name))))
    monkeypatch.setattr(b, "OUT_DIR", str(tmp_path))
    compiler = FakeCompiler()
    monkeypatch.setattr(b.subprocess, "Popen", compiler)
    monkeypatch.setattr(b.subprocess, "run", compiler)
    return compiler


def without_torch(monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def test_library_is_built_without_torch(fake, monkeypatch):
    without_torch(monkeypatch)
    assert b.build() == b.LIB_PATH and os.path.exists(b.LIB_PATH)
    assert "libw12.so" in fake.outputs() and "kv_host.so" not in fake.outputs()
    made = len(fake.commands)
    b.build()  # and is not stale for want of the module
    assert len(fake.commands) == made


def test_module_is_built_when_torch_appears(fake, monkeypatch):
    with monkeypatch.context() as m:
        without_torch(m)
        b.build()
    b.build()
    assert "kv_host.so" in fake.outputs() and os.path.exists(b.KV_HOST_PATH)
    made = len(fake.commands)
    b.build()
    assert len(fake.commands) == made


def test_module_is_built_again_for_another_torch(fake, tmp_path, monkeypatch):
    b.build()
    made = len(fake.commands)
    b.build()
    assert len(fake.commands) == made
    other = tmp_path / "elsewhere" / "torch"
    other.mkdir(parents=True)
    (other / "version.py").write_text("__version__ = '99.0'\n")
    find = importlib.util.find_spec

    class Spec:
        submodule_search_locations = [str(other)]

    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: Spec if name == "torch" else find(name, *a))
    b.build()
    assert "kv_host.so" in fake.outputs()[made:]
    made = len(fake.commands)
    (other / "version.py").write_text("__version__ = '99.1'\n")
    b.build()
    assert "kv_host.so" in fake.outputs()[made:]


HIDE = "import sys; sys.modules['torch'] = None\n"


@pytest.mark.parametrize("code", ["from lossless_bit_weight_encode_gb300 import *; print(W12Weight.__name__)",
                                  "from lossless_bit_weight_encode_gb300 import W12Weight; print(W12Weight.__name__)"])
def test_package_is_imported_without_torch(code):
    r = subprocess.run([sys.executable, "-c", HIDE + code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "W12Weight", r.stderr


def test_holders_are_imported_before_the_build(tmp_path):
    """Only a call needs the compiled module; without it the call says what to do."""
    code = ("from lossless_bit_weight_encode_gb300 import build\n"
            f"build.KV_HOST_PATH = {str(tmp_path / 'kv_host.so')!r}\n"
            "from lossless_bit_weight_encode_gb300 import *\n"
            "from lossless_bit_weight_encode_gb300 import kv\n"
            "print(KVCache.__name__, KVPages.__name__, KVStep.__name__)\n"
            "try:\n    kv._host.read()\nexcept RuntimeError as e:\n    print('build()' in str(e))\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.split() == ["KVCache", "KVPages", "KVStep", "True"], r.stderr
