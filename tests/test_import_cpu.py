"""What importing and building the package needs: the library alone. Without the extension module the
layer operators are called through ctypes; a PyTorch that is missing or broken is not needed for raw
addresses. Each import runs in an interpreter of its own, on a copy of the package. No GPU."""
import importlib.util
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "dense_gemm_tile_amd")


@pytest.fixture
def package(tmp_path):
    """A copy of the package without the extension module; what it prints for a program."""
    lib = os.path.join(PKG, "libdense_gemm_tile_amd.so")
    if not os.path.exists(lib):
        subprocess.run([sys.executable, os.path.join(PKG, "build.py")], check=True)
    copy = tmp_path / "dense_gemm_tile_amd"
    copy.mkdir()
    (copy / "__init__.py").write_text(open(os.path.join(PKG, "__init__.py")).read())
    os.symlink(lib, copy / "libdense_gemm_tile_amd.so")

    def run(program):
        done = subprocess.run([sys.executable, "-c", program], cwd=tmp_path, capture_output=True, text=True)
        assert done.returncode == 0, done.stderr
        return done.stdout.split()
    run.path = tmp_path
    return run


GEMM = ("import dense_gemm_tile_amd as dgt; A, B, D = 1 << 28, 2 << 28, 3 << 28; "
        "print(dgt.gemm_validate(8, 8, 8, 'bf16', 0, 1, 1.0, 0.0, A, 8, B, 8, None, 8, D, 8)); ")


def test_gemm_needs_no_extension_module(package):
    assert package(GEMM + "print(dgt.__file__)") == ["0", str(package.path / "dense_gemm_tile_amd" / "__init__.py")]


def test_a_broken_pytorch_is_not_needed(package):
    (package.path / "torch.py").write_text("raise RuntimeError('libtorch is of another version')\n")
    assert package(GEMM) == ["0"]
    (package.path / "torch.py").write_text("raise OSError('libtorch.so: cannot open shared object file')\n")
    assert package(GEMM) == ["0"]


# Refused and empty calls of every entry point: (name, arguments before the stream). Tensors are T(address).
CALLS = """
A, B, C, D, E, F = (T(i << 28) for i in range(1, 7))
calls = [
    ("gemm_linear", (8, 8, 8, "bf16", 0, 1, A, 8, B, 8, None, "gelu", None, 0, A, 8, "bf16", None, 0)),
    ("gemm_linear", (0, 8, 8, 1, False, True, A, 8, B, 8, C, 4, D, 8, E, 8, "f32", F, 8)),
    ("gemm_linear", (8, 8, 8, "f16", 0, 1, A, 7, B, 8, None, "none", None, 0, D, 8, "f16", None, 0)),
    ("gemm_linear", (8, 8, 8, "swish", 0, 1, A, 8, B, 8, None, "gelu", None, 0, D, 8, "bf16", None, 0)),
    ("gemm_linear", (8, 8, 8, "bf16", 0, 1, A, 8, B, 8, None, "f16", None, 0, D, 8, "bf16", None, 0)),
    ("gemm_linear", (8, 8, 8, "bf16", 0, 1, A, 8, B, 8, None, "none", None, 0, D, 8, "relu", None, 0)),
    ("gemm_grouped", (4, 0, 8, 8, "f16", 1, E, A, 8, B, 8, 64, C, "silu", None, 0, D, 8, "f32", F, 8)),
    ("gemm_grouped", (4, 8, 8, 8, "f16", 1, None, A, 8, B, 8, 64, C, "silu", None, 0, D, 8, "f32", F, 8)),
    ("gemm_grouped_grad_weight", (0, 8, 8, 8, "f16", E, A, 8, B, 8, D, 8, 64, "f32", True)),
    ("gemm_grouped_grad_weight", (2, 8, 8, 8, "f16", E, A, 8, B, 8, D, 8, 63, "f16", False)),
    ("gemm_act_grad", (1, 0, 8, "bf16", "gelu_erf", None, A, 8, B, 8, D, 8, None, None, 0)),
    ("gemm_act_grad", (1, 8, 8, "bf16", "relu", None, A, 8, B, 8, D, 8, E, F, 0)),
    ("gemm_route", (8, 2, 2000, A, B, C, D, None, 0)),
    ("gemm_dispatch", (0, 2, 8, "f32", A, 8, B, C, 8)),
    ("gemm_dispatch", (4, 2, 8, "f32", A, 8, B, A, 8)),
    ("gemm_combine", (0, 2, 8, "bf16", A, 8, B, C, D, 8, E, 8)),
    ("gemm_combine", (4, 2, 8, "bf16", A, 8, B, C, D, 7, E, 8)),
    ("gemm_combine_grad", (0, 2, 8, "f16", A, 8, B, 8, C, D, E, 8, F)),
    ("gemm_combine_grad", (4, 2, 8, "f16", A, 8, B, 8, C, D, E, 8, B)),
]
"""
SHOW = """
class T:
    def __init__(self, at): self.at = at
    def data_ptr(self): return self.at
class S: cuda_stream = 0
import dense_gemm_tile_amd as dgt
""" + CALLS + """
for name, args in calls:
    for stream in (None, 0, S()):
        try:
            getattr(dgt, name)(*args, stream=stream)
            print(name, 0)
        except dgt.GemmError as e:
            print(name, e.code, dgt.gemm_last_error().replace(" ", "_"))
        except KeyError as e:
            print(name, "KeyError", e.args[0])
print(dgt.gemm_route_workspace(70000, 4, 64), dgt.gemm_act_grad_workspace(3, 100, 64))
"""


def test_layer_operators_without_the_extension_module(package):
    with_module = subprocess.run([sys.executable, "-c", SHOW], cwd=ROOT, capture_output=True, text=True, check=True)
    assert package(SHOW) == with_module.stdout.split()
    assert {"0", "1", "2", "3", "KeyError"} <= set(package(SHOW))


def test_a_build_without_python_headers_leaves_the_module_out(tmp_path, monkeypatch, capsys):
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(PKG, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    stale = tmp_path / "_binding.so"
    stale.write_text("")
    monkeypatch.setattr(build, "BINDING_PATH", str(stale))
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    build._build_binding()
    assert not stale.exists() and "Python.h" in capsys.readouterr().err
