"""The build without torch, and with a binding module that does not compile
(CPU only; one small source in place of the library's)."""
import os
import subprocess
import sys

import pytest

from paged_kv_cache_varlen_gb300 import build

CODE = """
import importlib.util, os, sys
spec = importlib.util.spec_from_file_location("pkv_build", sys.argv[1])
build = importlib.util.module_from_spec(spec)
spec.loader.exec_module(build)
out = sys.argv[2]
build.BUILD_DIR = os.path.join(out, "objects")
build.LIBRARY = os.path.join(out, "libpkv.so")
build.MARSHAL = os.path.join(out, "_marshal.so")
build.SOURCES = ["block_manager.cpp"]
if sys.argv[3] == "no torch":
    sys.modules["torch"] = None
else:
    build._torch_paths = lambda: (["-include", "/no/such/header.h"], "/no/such/folder")
print(build.build(force=True))
print("up to date:", build.up_to_date())
"""


def run(tmp_path, what):
    return subprocess.run([sys.executable, "-c", CODE, build.__file__, str(tmp_path), what],
                          capture_output=True, text=True, timeout=300)


def test_the_library_needs_no_torch(tmp_path):
    r = run(tmp_path, "no torch")
    assert r.returncode == 0, r.stderr
    assert os.path.exists(tmp_path / "libpkv.so") and not os.path.exists(tmp_path / "_marshal.so")
    assert "up to date: True" in r.stdout


def test_a_binding_module_that_does_not_compile_is_an_error_beside_the_library(tmp_path):
    r = run(tmp_path, "bad headers")
    assert r.returncode != 0 and "marshal.cpp" in r.stderr
    assert os.path.exists(tmp_path / "libpkv.so")


@pytest.mark.parametrize("missing", ["LIBRARY", "MARSHAL"])
def test_a_build_without_either_part_is_out_of_date(tmp_path, monkeypatch, missing):
    for name in ("LIBRARY", "MARSHAL"):
        path = tmp_path / name
        path.write_bytes(b"")
        monkeypatch.setattr(build, name, str(path))
    assert build.up_to_date()
    os.remove(tmp_path / missing)
    assert not build.up_to_date()
