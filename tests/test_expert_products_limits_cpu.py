"""Refusals of the 16-bit and int8 expert products and their gradients that concern sizes and memory: every call below
fails validation before anything is enqueued."""
import ctypes

import pytest

import indirect_expert_matmul_amd as moe

AT = 1 << 44   # never dereferenced


def _product(rows, T, k, E=8, typ=moe.MOE_BF16, cols=16, weighted=False, path=0, B=1):
    w = moe.c_moe_weights(typ, AT, AT if typ == moe.MOE_I8 else None, E, rows, cols)
    opt = moe._options(path)
    return moe.lib.moe_mul_mat_id(ctypes.byref(w), AT, moe.MOE_BF16, B, AT, T, k, AT if weighted else None, AT,
                                  ctypes.byref(opt), AT, 1 << 50, None)


@pytest.mark.parametrize("typ", [moe.MOE_BF16, moe.MOE_I8])
def test_gemv_of_more_rows_than_a_dispatch_holds(typ):
    """Four rows a wave: 2^28 rows are 2^32 work-items."""
    for T, k, weighted in ((1, 1, False), (1, 8, True), (8, 4, False), (8, 4, True)):
        for path in (0, 2):
            assert _product(1 << 28, T, k, typ=typ, weighted=weighted, path=path) == moe.MOE_ELIMIT
            assert "work-items" in moe.last_error()
