"""The binding's native part: the rest of the package works without it, and the build notices when it
was made for another torch or Python.  No GPU needed."""

import importlib.util
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = """
import sys
sys.modules["tiled_dense_gemm_tlg_b200._binding"] = None  # as a missing file: its import fails
import torch
import tiled_dense_gemm_tlg_b200 as tlg
A = torch.zeros((8, 8), dtype=torch.float16)
try:
    tlg.tlg_gemm_f16f32(A, A)
except tlg.TlgError as e:  # the library's answer to host memory
    print("refused by the library")
assert tlg.tlg_mx_size("e2m1", 1, 64) == (32, 512)
for call in (lambda: tlg.tlg_mx_quantize(A), lambda: tlg.tlg_act_forward_mx(A, "gelu")):
    try:
        call()
    except ImportError as e:
        print("ImportError", "build.py" in str(e), e.__cause__ is not None)
"""


@pytest.fixture(scope="module")
def build():
    spec = importlib.util.spec_from_file_location("tlg_build",
                                                  os.path.join(ROOT, "tiled_dense_gemm_tlg_b200", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.build()
    return mod


def test_the_package_imports_without_the_binding(build):
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split("\n")[:3] == ["refused by the library"] + 2 * ["ImportError True True"]


def test_the_build_notices_another_torch(build, monkeypatch):
    assert not build.binding_needs_build()
    import tiled_dense_gemm_tlg_b200 as tlg
    assert tlg._binding.__doc__ == build.binding_built_for()
    from importlib import metadata
    monkeypatch.setattr(metadata, "version", lambda name: "1.0")
    assert build.binding_needs_build()


def test_a_torch_that_is_no_installed_package(build, monkeypatch):
    from importlib import metadata

    import torch

    def missing(name):
        raise metadata.PackageNotFoundError(name)

    monkeypatch.setattr(metadata, "version", missing)
    assert f"torch {torch.__version__}," in build.binding_built_for()
