"""The native binding of the paged-cache calls, as far as it goes without a GPU."""
from __future__ import annotations

import pytest
import torch

import softmax_learned_covariance_b200 as plx


def cpu_cache():
    """(q, codes, exponents, table, seqlens) on the CPU: refused, but only after the other arguments are read."""
    codes = torch.zeros((4, 2, 16, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    table, sl = torch.zeros((1, 2), dtype=torch.int32), torch.zeros((1,), dtype=torch.int32)
    return torch.zeros((1, 2, 64), dtype=torch.bfloat16), codes, torch.zeros((4, 2, 1), dtype=torch.int8), table, sl


def test_an_error_of_want_lse_is_the_callers():
    """An object without a truth value: its own error, not a result with an error set beside it."""
    class Neither:
        def __bool__(self):
            raise ArithmeticError("neither true nor false")

    q, codes, e, table, sl = cpu_cache()
    with pytest.raises(ArithmeticError):
        plx.parallax_decode_paged_q8(q, None, codes, codes, e, e, table, sl, want_lse=Neither())
