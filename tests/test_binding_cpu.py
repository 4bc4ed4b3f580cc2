"""The extension module that calls the layer operators' entry points: argument conversion and the
status codes, against the same calls through ctypes. No GPU: every call here is refused or does
nothing."""
import ctypes

import pytest

import dense_gemm_tile_amd as dgt
from dense_gemm_tile_amd import _binding

A0, B0, Y0 = 0x10000000, 0x20000000, 0x30000000


class Tensor:
    def __init__(self, at):
        self.at = at

    def data_ptr(self):
        return self.at


class Stream:
    cuda_stream = 0


def combine(T=0, top=2, H=64, dtype="bf16", ys=A0, ldys=64, slot=B0, w=None, r=None, ldr=0, y=Y0, ldy=64, stream=None):
    return T, top, H, dtype, ys, ldys, slot, w, r, ldr, y, ldy, stream


def test_every_argument_form_of_a_pointer_and_a_stream():
    for ys in (None, A0, Tensor(A0), 2 ** 63 + 5):
        for stream in (None, 0, Stream()):
            assert _binding.gemm_combine(*combine(ys=ys, stream=stream)) == 0


def test_status_codes_are_the_library_s():
    calls = [combine(), combine(T=-1), combine(T=4, ldys=3), combine(T=4, dtype=9), combine(T=4, y=None),
             combine(T=4, y=A0), combine(T=4, r=Y0 + 64, ldr=64), combine(T=2 ** 40), combine(T=4, dtype=4),
             combine(T=4, slot=B0 + 2)]
    for c in calls:
        T, top, H, dtype, ys, ldys, slot, w, r, ldr, y, ldy, _ = c
        code = {"bf16": 1}.get(dtype, dtype)
        want = dgt._lib.gemm_combine(T, top, H, code, ys, ldys, slot, w, r, ldr, y, ldy, None)
        message = dgt.gemm_last_error()
        assert _binding.gemm_combine(*c) == want
        assert dgt.gemm_last_error() == message
    assert {dgt._lib.gemm_combine(c[0], c[1], c[2], 1, *c[4:12], None) for c in calls} >= {0, 1, 2, 3}


def test_names_and_codes_of_types_and_activations():
    for name, code in (("f16", 0), ("bf16", 1), ("f32", 6)):
        assert _binding.gemm_combine(*combine(dtype=name)) == _binding.gemm_combine(*combine(dtype=code)) == 0
    for act, code in (("none", 0), ("relu", 1), ("gelu", 2), ("gelu_erf", 3), ("silu", 4)):
        for a in (act, code):
            assert _binding.gemm_act_grad(1, 0, 8, "f16", a, None, A0, 8, B0, 8, Y0, 8, None, None, 0, None) == 0
    assert _binding.gemm_act_grad(1, 4, 8, "f16", 5, None, A0, 8, B0, 8, Y0, 8, None, None, 0, None) == 1
    with pytest.raises(KeyError):
        _binding.gemm_combine(*combine(dtype="int3"))
    with pytest.raises(KeyError):
        _binding.gemm_act_grad(1, 0, 8, "f16", "swish", None, A0, 8, B0, 8, Y0, 8, None, None, 0, None)


def test_what_cannot_be_converted_raises():
    for bad in (combine(T="4"), combine(T=4.5), combine(ys="x"), combine(ys=1.5), combine(stream="s"),
                combine(dtype=1.5)):
        with pytest.raises((TypeError, AttributeError)):
            _binding.gemm_combine(*bad)
    with pytest.raises(OverflowError):
        _binding.gemm_combine(*combine(T=2 ** 63))
    with pytest.raises(OverflowError):
        _binding.gemm_combine(*combine(dtype=2 ** 40))
    with pytest.raises(TypeError):
        _binding.gemm_combine(*combine()[:-1])
    with pytest.raises(TypeError):
        _binding.gemm_combine(*combine(), None)


def test_an_exception_of_data_ptr_passes_through():
    class Broken:
        def data_ptr(self):
            raise RuntimeError("gone")

    with pytest.raises(RuntimeError, match="gone"):
        _binding.gemm_combine(*combine(ys=Broken()))


def test_workspace_sizes():
    assert _binding.gemm_route_workspace(70000, 4, 64) == dgt._lib.gemm_route_workspace(70000, 4, 64) > 0
    assert _binding.gemm_act_grad_workspace(3, 100, 64) == dgt._lib.gemm_act_grad_workspace(3, 100, 64) > 0
    assert isinstance(_binding.gemm_route_workspace(1, 1, 1), int)


def test_every_enqueueing_entry_point_of_the_header_is_there():
    names = {n for n in dgt._SIGNATURES if n.startswith("gemm_") and not n.endswith("_validate")}
    layer = names - {"gemm_i8", "gemm_last_error", "gemm_last_path", "gemm_tile_order"}
    assert layer <= {n for n in dir(_binding) if n.startswith("gemm_")}
    assert ctypes.sizeof(ctypes.c_void_p) == 8


def test_the_package_may_be_imported_first():
    """PyTorch's HIP runtime is loaded before the library's, whichever the program imports first."""
    import subprocess
    import sys
    out = subprocess.run([sys.executable, "-c", "import dense_gemm_tile_amd, sys; print('torch' in sys.modules); "
                          "import torch; m = [l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l]; "
                          "print(len(set(m)))"], capture_output=True, text=True, check=True,
                         cwd=__file__.rsplit("/tests/", 1)[0])
    assert out.stdout.split()[0] == "True", out.stdout
