"""``libcpattn.so`` and ``_binding.so`` apart: most calls need the former alone, and
the latter is bound to one PyTorch."""

import os
import shutil
import subprocess
import sys

import pytest

from long_context_gb300 import build as lib_build

SCRIPT = """
import torch
from long_context_gb300 import cpattn
assert cpattn.plan([100, 5000, 30], 4, 4096, 4)["num_micro_batches"] >= 1
assert cpattn.workspace_size(1000, 1, 8, 64, 1) > 0
assert cpattn.paged_workspace_size(4, 2, 8, 4, 64, 2) > 0
q = torch.zeros(4, 8, 64, dtype=torch.bfloat16)
try:
    cpattn.qk_norm_rope(q, q, torch.zeros(4, dtype=torch.int32), torch.zeros(8, 64))
except ImportError as e:
    assert "_binding.so" in str(e) and "build()" in str(e)
else:
    raise SystemExit("no ImportError")
"""


@pytest.mark.parametrize("binding", ["missing", "of another build"])
def test_calls_that_need_the_library_alone(tmp_path, binding):
    lib_build.build()
    pkg = tmp_path / "long_context_gb300"
    pkg.mkdir()
    for name in os.listdir(lib_build.PKG):
        if name.endswith(".py") or name == "libcpattn.so":
            shutil.copy(os.path.join(lib_build.PKG, name), pkg)
    if binding != "missing":
        (pkg / "_binding.so").write_bytes(b"no library that this process can load")
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=tmp_path, capture_output=True,
                       text=True, env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode == 0, r.stdout + r.stderr


def _torch(root, version, cuda=True):
    (root / "lib").mkdir(parents=True)
    if cuda:
        (root / "lib" / "libc10_cuda.so").write_bytes(b"")
    f = root / "version.py"
    f.write_text("__version__ = %r\n" % version)
    os.utime(f, (1e9, 1e9))  # installed long before the binding was built
    return str(root)


def test_another_pytorch_makes_the_binding_stale(monkeypatch, tmp_path):
    lib_build.build()
    assert not lib_build._binding_stale()
    other = _torch(tmp_path / "a", "1.2.3")
    monkeypatch.setattr(lib_build, "_torch_dir", lambda: other)
    assert lib_build._binding_stale()


@pytest.mark.parametrize("installed", [False, True])
def test_build_without_cuda_in_pytorch(monkeypatch, tmp_path, installed):
    """No PyTorch, or one without CUDA: the library is built, the binding is not."""
    lib_build.build()
    root = _torch(tmp_path / "b", "1.2.3+cpu", cuda=False) if installed else None
    monkeypatch.setattr(lib_build, "_torch_dir", lambda: root)
    monkeypatch.setattr(lib_build, "BINDING", str(tmp_path / "_binding.so"))
    assert lib_build.build() == lib_build.LIB
    assert not os.path.exists(lib_build.BINDING)


def test_an_error_of_the_binding_leaves_the_library(monkeypatch, tmp_path):
    for name, value in (("BUILD", tmp_path), ("LIB", tmp_path / "libcpattn.so"),
                        ("BINDING", tmp_path / "_binding.so"),
                        ("BINDING_FOR", tmp_path / "binding.for")):
        monkeypatch.setattr(lib_build, name, str(value), raising=False)
    monkeypatch.setattr(lib_build, "SOURCES", ["plan.cpp"])

    def fail():
        raise RuntimeError("g++ binding.cpp failed")

    monkeypatch.setattr(lib_build, "_compile_binding", fail)
    with pytest.raises(RuntimeError, match="binding.cpp"):
        lib_build.build()
    assert os.path.exists(lib_build.LIB)
