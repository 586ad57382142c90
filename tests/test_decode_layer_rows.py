"""Without a GPU: rows of heads where the call has one row, and the binding's two call paths."""
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
