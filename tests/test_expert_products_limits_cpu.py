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


T, K_USED, E, N, K = 64, 2, 8, 64, 128
MB = 1 << 20


def _backward(B=1, ws=1 << 50, **at):
    """Every tensor a megabyte from the next one, but for those named."""
    names = ("src1", "ids", "route_w", "d_dst", "w", "d_src1", "d_w", "d_route_w", "ws")
    p = {n: AT + i * MB for i, n in enumerate(names)}
    p.update(at)
    w = moe.c_moe_weights(moe.MOE_BF16, p["w"], None, E, N, K)
    opt = moe._options(0)
    return moe.lib.moe_mul_mat_id_backward(ctypes.byref(w), p["src1"], moe.MOE_BF16, B, p["ids"], T, K_USED, p["route_w"],
                                           p["d_dst"], moe.MOE_BF16, p["d_src1"], p["d_w"], moe.MOE_BF16, p["d_route_w"],
                                           ctypes.byref(opt), p["ws"], ws, None)


BYTES = dict(src1=T * K * 2, ids=T * K_USED * 4, route_w=T * K_USED * 4, d_dst=T * N * 2, w=E * N * K * 2, d_src1=T * K * 2,
             d_w=E * N * K * 2, d_route_w=T * K_USED * 4)


def test_gradients_that_overlap():
    """Outputs that share memory with an input, or another output, wherever they begin."""
    start = {n: AT + i * MB for i, n in enumerate(("src1", "ids", "route_w", "d_dst", "w", "d_src1", "d_w", "d_route_w"))}
    for out in ("d_src1", "d_w", "d_route_w"):
        for other in start:
            if other == out:
                continue
            for at in (start[other], start[other] + BYTES[other] - 16, start[other] - BYTES[out] + 16):
                assert _backward(**{out: at}) == moe.MOE_EINVAL, (out, other)
                assert "inputs" in moe.last_error() or "overlap" in moe.last_error()


def test_quantizer_that_overlaps():
    f = moe.lib.moe_quantize_rows
    x, q, d = AT, AT + MB, AT + 2 * MB
    rows, cols = 100, 50
    for typ, size in ((moe.MOE_F32, 4), (moe.MOE_BF16, 2)):
        for a, b in ((x + rows * cols * size - 4, d), (x - rows * cols + 1, d), (q, x + 4), (q, x - 4), (q, q + rows * cols - 1 & ~3),
                     (q, q - 4 * rows + 4)):
            assert f(x, typ, rows, cols, a, b, None) == moe.MOE_EINVAL and "overlap" in moe.last_error()
    assert f(x, moe.MOE_F32, 1 << 40, 1 << 30, q, d, None) == moe.MOE_ELIMIT
