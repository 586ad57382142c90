"""Without a GPU: rows of heads where the call has one row, and the two call paths of the binding."""
import subprocess
import sys

import pytest

from tests.test_decode_layer_host import GOOD, bz  # noqa: F401

ROOT = __file__.rsplit("/", 2)[0]


def test_one_row_of_a_wider_matrix_keeps_its_stride(bz):  # noqa: F811
    """A slice of one row counts as contiguous; its stride is the matrix's all the same."""
    import torch

    def ld(t, rows, width):
        return bz._rows(t, rows, width, None, -1)[1]
    for T in (1, 2, 5):
        qkv = torch.zeros(T, 448, dtype=torch.float16)
        assert ld(qkv, T, 448) == 448
        assert ld(qkv[:, :256], T, 256) == 448
        assert ld(qkv[:, 256:384], T, 128) == 448
    assert ld(torch.zeros(4, 448, dtype=torch.float16)[:1, :256], 1, 256) == 448
    # a stride that no second row uses, and that rows could not have
    odd = torch.zeros(1000, dtype=torch.float16)
    assert ld(odd.as_strided((1, 256), (1, 1)), 1, 256) == 256
    assert ld(odd.as_strided((1, 256), (300, 1)), 1, 256) == 256  # not a multiple of 8
    assert ld(odd.as_strided((1, 256), (304, 1)), 1, 256) == 304


def test_in_place_strides_of_one_row_are_not_compared(bz):  # noqa: F811
    """With one row there is no second one to start elsewhere.  (The pointer of the frequencies is
    unaligned, the check after the one in question: nothing is launched.)"""
    def rope(T):
        return bz.raw().bonsai_rope(GOOD, GOOD, GOOD + 4, GOOD, T, 2, 64, 64, 448, 128, 1.0, 0, None)

    def append(T):
        return bz.raw().bonsai_rope_append(GOOD, GOOD, 2 * GOOD, 3 * GOOD, None, None, GOOD + 4, GOOD, GOOD, T, 4, 2, 64, 64,
                                           512, 256, 8, 16, 1.0, 0, 0, None)
    assert rope(2) == append(2) == bz.BONSAI_ERR_SHAPE
    assert rope(1) == append(1) == bz.BONSAI_ERR_ALIGN


CALLS = ["bonsai_ternary_linear", "bonsai_ternary_linear_swiglu", "bonsai_ternary_linear_epilogue", "bonsai_rope",
         "bonsai_rope_append", "bonsai_paged_attention"]

WITHOUT = """
import sys
sys.modules["ternary_weight_02_b200._bonsai_call"] = None  # an import of it fails
from ternary_weight_02_b200 import bonsai as bz
assert bz._call is bz.raw()
G = 1 << 20
for call in (lambda: bz.bonsai_ternary_linear(None, G, G, G, 1, 8, 128, 2, stream=0),
             lambda: bz.bonsai_ternary_linear_swiglu(None, G, G, G, 1, 8, 128, 2, stream=0)):
    try:
        call()
    except bz.BonsaiError as e:
        assert e.status == bz.BONSAI_ERR_NULL
    else:
        raise AssertionError
"""


def test_binding_without_its_extension_module():
    res = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


def test_both_call_paths_take_the_same_arguments(bz):  # noqa: F811
    """Each entry point refuses the same arguments with the same status through both."""
    from ternary_weight_02_b200 import _bonsai_call as fast
    args = {"bonsai_ternary_linear": (GOOD, GOOD, None, GOOD, 1, 8, 128, 2, None),
            "bonsai_ternary_linear_swiglu": (GOOD, GOOD, GOOD, GOOD + 2, 1, 8, 128, 2, 0),
            "bonsai_ternary_linear_epilogue": (GOOD, GOOD, GOOD, None, None, GOOD, 1, 8, 128, 2, 7, 0, 0, None),
            "bonsai_rope": (GOOD, GOOD, GOOD, GOOD, 4, 2, 64, 66, 128, 128, 1.0, 0, None),
            "bonsai_rope_append": (GOOD, 2 * GOOD, GOOD, GOOD, None, None, GOOD, GOOD, GOOD, 4, 4, 2, 64, 64, 512, 256, 8, 16,
                                   0.5, 0, 1, None),
            "bonsai_paged_attention": (GOOD, GOOD, GOOD, None, None, GOOD, GOOD, GOOD, None, 2, 4, 2, 64, 256, 256, 8, 16, 4, -1,
                                       1.0, 0, None)}
    assert sorted(args) == sorted(CALLS)
    for name, a in args.items():
        slow = getattr(bz.raw(), name)(*a)
        assert slow < 0 and getattr(fast, name)(*a) == slow, name
        with pytest.raises(TypeError):
            getattr(fast, name)(*a[:-1])


def test_build_without_a_c_compiler(bz, monkeypatch, tmp_path, capsys):  # noqa: F811
    """The library's build goes on without the extension module, and says so."""
    from ternary_weight_02_b200 import build
    monkeypatch.setenv("CC", str(tmp_path / "no-such-compiler"))
    monkeypatch.setattr(build, "CALL", str(tmp_path / "_bonsai_call.abi3.so"))
    assert build.build_call() is None
    assert "ctypes" in capsys.readouterr().err
    assert build.build() == build.LIB
