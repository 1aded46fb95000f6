"""The build script without a compiler run: what is built where torch is
missing or another one than the binding was built against."""
import subprocess
import sys

import pytest

_WITHOUT_TORCH = """
import sys
sys.modules["torch"] = None
from head_wise_kv_b200 import build
build.BINDING = sys.argv[1]             # not there yet
assert build.build() == build.LIB
assert "torch" not in [m for m, v in sys.modules.items() if v is not None]
"""


def _up_to_date():
    import os
    from head_wise_kv_b200 import build
    if not os.path.exists(build.LIB) or not os.path.isdir(build.OBJDIR):
        pytest.skip("nothing built here")


def test_the_library_builds_without_torch(tmp_path):
    _up_to_date()
    done = subprocess.run([sys.executable, "-c", _WITHOUT_TORCH, str(tmp_path / "_binding.so")], capture_output=True, text=True,
                          timeout=600)
    assert done.returncode == 0, done.stderr[-2000:]
    assert "C library alone" in done.stderr and not (tmp_path / "_binding.so").exists()


def test_another_torch_or_python_rebuilds_the_binding(tmp_path, monkeypatch):
    from head_wise_kv_b200 import build
    ran = []
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build, "BUILT_FOR", str(tmp_path / "built_for"))
    monkeypatch.setattr(build, "OBJDIR", str(tmp_path))
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, check: (ran.append(cmd), open(build.BINDING, "w").close()))
    build.build_binding()
    build.build_binding()
    assert len(ran) == 1
    monkeypatch.setattr(build, "built_for", lambda: "python 3.99\ntorch 9.9\n")
    build.build_binding()
    build.build_binding()
    assert len(ran) == 2
    build.build_binding(force=True)
    assert len(ran) == 3
