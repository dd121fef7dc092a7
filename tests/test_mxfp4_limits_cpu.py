"""The documented limits of MXFP4 activations hold on both paths: refused before any HIP call."""
import ctypes

import pytest

import indirect_expert_matmul_amd as moe

FAKE = 0x10000  # never dereferenced: every call below fails validation first


@pytest.mark.parametrize("path", [moe.PATH_GEMV, moe.PATH_GEMM])
def test_cols_limit(path):
    def w(n_mat, rows, cols):
        return moe.c_moe_weights(moe.MOE_MXFP4, FAKE, FAKE, n_mat, rows, cols)
    opt = moe._options(path, act_quant=2)
    for cols in (1 << 24, 1 << 26, (1 << 31) - 32):
        m = w(2, 64, cols)
        for route_w in (None, FAKE):
            assert moe.lib.moe_mul_mat_id(ctypes.byref(m), FAKE, moe.MOE_BF16, 1, FAKE, 1, 1, route_w, FAKE,
                                          ctypes.byref(opt), FAKE, 1 << 60, None) == moe.MOE_ELIMIT
            assert "2^24" in moe.last_error()
        for n_embd, n_ff in ((cols, 128), (128, cols)):
            g, d = w(2, n_ff, n_embd), w(2, n_embd, n_ff)
            sg, sd = w(1, 128, 128), w(1, 128, 128)
            r = ctypes.byref
            assert moe.lib.moe_ffn_fused(r(g), r(g), r(d), None, None, None, FAKE, moe.MOE_BF16, FAKE, FAKE, 1, 1,
                                         FAKE, r(opt), FAKE, 1 << 60, None) == moe.MOE_ELIMIT
            assert "2^24" in moe.last_error()
        g, sg, sd = w(2, 128, 128), w(1, cols, 128), w(1, 128, cols)   # shared experts alone too wide
        assert moe.lib.moe_ffn_fused(r(g), r(g), r(g), r(sg), r(sg), r(sd), FAKE, moe.MOE_BF16, FAKE, FAKE, 1, 1,
                                     FAKE, r(opt), FAKE, 1 << 60, None) == moe.MOE_ELIMIT
        assert "2^24" in moe.last_error()


@pytest.mark.parametrize("path", [moe.PATH_GEMV, moe.PATH_GEMM])
def test_rows_limit(path):
    """Row numbers past the last row, up to a whole tile, must not leave int32."""
    opt = moe._options(path, act_quant=2)
    for rows in ((1 << 31) - 1, (1 << 31) - 512):
        m = moe.c_moe_weights(moe.MOE_MXFP4, FAKE, FAKE, 1, rows, 128)
        assert moe.lib.moe_mul_mat_id(ctypes.byref(m), FAKE, moe.MOE_BF16, 1, FAKE, 1, 1, None, FAKE,
                                      ctypes.byref(opt), FAKE, 1 << 60, None) == moe.MOE_ELIMIT
        assert "2^31" in moe.last_error()


@pytest.mark.parametrize("path", [moe.PATH_GEMV, moe.PATH_GEMM])
def test_workspace_alignment(path):
    """The codes of activations and of h lie in the workspace and are copied 16 bytes at a time."""
    m = moe.c_moe_weights(moe.MOE_MXFP4, FAKE, FAKE, 4, 128, 128)
    opt, r = moe._options(path, act_quant=2), ctypes.byref
    for off in (1, 4, 8):
        assert moe.lib.moe_mul_mat_id(r(m), FAKE, moe.MOE_BF16, 1, FAKE, 9, 2, FAKE, FAKE, r(opt), FAKE + off, 1 << 40,
                                      None) == moe.MOE_EINVAL
        assert "workspace" in moe.last_error()
        assert moe.lib.moe_ffn_fused(r(m), r(m), r(m), None, None, None, FAKE, moe.MOE_BF16, FAKE, FAKE, 9, 2, FAKE,
                                     r(opt), FAKE + off, 1 << 40, None) == moe.MOE_EINVAL
        assert "workspace" in moe.last_error()
