"""CPU checks for the 16-bit and int8 expert products: the float64 forms that the GPU tests compare
against are pinned to autograd and to differences, and the library refuses bad arguments before any
HIP call."""
import ctypes

import pytest
import torch

import indirect_expert_matmul_amd as moe
import ref_products as ref

FAKE = 0x10000  # never dereferenced: every call below fails validation first


# ---------------------------------------------------------------- the float64 forms
@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_gradients_match_autograd_and_differences(per_slot, weighted):
    T, E, k, N, K = 5, 4, 3, 6, 8
    g = torch.Generator().manual_seed(1)
    ids = torch.rand((T, E), generator=g).topk(k, 1).indices.int()
    ids[1, 0], ids[4, 2] = -1, E
    w = torch.randn((E, N, K), generator=g, dtype=torch.float64).requires_grad_(True)
    x = torch.randn((T * (k if per_slot else 1), K), generator=g, dtype=torch.float64).requires_grad_(True)
    rw = torch.rand((T, k), generator=g).double().requires_grad_(True)
    dy = torch.randn((T, N) if weighted else (T, k, N), generator=g, dtype=torch.float64)

    def loss(w, x, rw):
        total = 0.0
        for t in range(T):
            for s in range(k):
                e = int(ids[t, s])
                if 0 <= e < E:
                    y = w[e] @ x[t * k + s if per_slot else t]
                    total = total + ((rw[t, s] * y * dy[t]).sum() if weighted else (y * dy[t, s]).sum())
        return total
    loss(w, x, rw).backward()
    got = ref.grads(w.detach(), x.detach(), ids, dy, rw.detach() if weighted else None, per_slot,
                    torch.float32, torch.float32)
    assert torch.allclose(got[0][0], x.grad, rtol=1e-12, atol=1e-14)
    assert torch.allclose(got[1][0], w.grad, rtol=1e-12, atol=1e-14)
    if weighted:
        assert torch.allclose(got[2][0], rw.grad, rtol=1e-12, atol=1e-14)
    with torch.no_grad():
        for p, d, at in ((w, got[1][0], (2, 3, 5)), (x, got[0][0], (2, 1))):
            a, b = p.clone(), p.clone()
            a[at] += 1e-6
            b[at] -= 1e-6
            lo, hi = ((loss(b, x, rw), loss(a, x, rw)) if p is w else (loss(w, b, rw), loss(w, a, rw)))
            assert abs((hi - lo) / 2e-6 - d[at]) < 1e-7


def test_quantize_rows_by_hand():
    x = torch.tensor([[127.0, 63.5, -62.5, 0.4], [0, 0, 0, 0], [1.0, -2.0, 0.5, float("inf")]])
    q, d = ref.quantize_rows(x)
    assert q[0].tolist() == [127, 64, -62, 0] and d[0] == 1
    assert q[1].tolist() == [0, 0, 0, 0] and d[1] == 0
    assert q[2].tolist() == [0, 0, 0, 0] and torch.isnan(d[2])


def test_product_is_the_dense_one():
    g = torch.Generator().manual_seed(2)
    ids = torch.tensor([[0, 2], [1, -1]], dtype=torch.int32)
    w, x = torch.randn((3, 4, 8), generator=g).double(), torch.randn((2, 8), generator=g).double()
    y, _ = ref.product(w, x, ids, 3, False)
    assert torch.allclose(y[0], w[0] @ x[0]) and torch.allclose(y[1], w[2] @ x[0])
    assert torch.allclose(y[2], w[1] @ x[1]) and (y[3] == 0).all()


# ---------------------------------------------------------------- refusals
def _w(typ=moe.MOE_BF16, n_mat=8, rows=64, cols=128, data=FAKE, scales=FAKE):
    return moe.c_moe_weights(typ, data, scales if typ == moe.MOE_I8 else None, n_mat, rows, cols)


def _mm(w=None, st=moe.MOE_BF16, path=0, aq=0, ws=1 << 40, x=FAKE, T=64, k=2, B=1, wsp=FAKE, rw=None):
    opt = moe._options(path, act_quant=aq)
    return moe.lib.moe_mul_mat_id(ctypes.byref(w or _w()), x, st, B, FAKE, T, k, rw, FAKE, ctypes.byref(opt), wsp,
                                  ws, None)


def test_product_validation():
    assert _mm(ws=16) == moe.MOE_EWORKSPACE                # valid up to the workspace
    assert _mm(_w(moe.MOE_F16), st=moe.MOE_F16, ws=16) == moe.MOE_EWORKSPACE
    for st in (moe.MOE_BF16, moe.MOE_F16, moe.MOE_F32):
        assert _mm(_w(moe.MOE_I8), st=st, ws=16) == moe.MOE_EWORKSPACE
    assert _mm(st=moe.MOE_F16) == moe.MOE_EINVAL and "BF16" in moe.last_error()
    assert _mm(_w(moe.MOE_F16)) == moe.MOE_EINVAL
    assert _mm(st=moe.MOE_F32) == moe.MOE_EINVAL
    assert _mm(_w(moe.MOE_I8), st=moe.MOE_I8) == moe.MOE_EINVAL
    assert _mm(_w(cols=100)) == moe.MOE_ELIMIT
    assert _mm(_w(moe.MOE_I8, cols=72)) == moe.MOE_ELIMIT
    assert _mm(_w(moe.MOE_I8, cols=131088)) == moe.MOE_ELIMIT
    assert _mm(_w(moe.MOE_I8, cols=131072), ws=16) == moe.MOE_EWORKSPACE
    assert _mm(_w(rows=1 << 30)) == moe.MOE_ELIMIT
    assert _mm(_w(cols=1 << 30)) == moe.MOE_ELIMIT
    assert _mm(_w(data=FAKE + 8)) == moe.MOE_EINVAL
    assert _mm(x=FAKE + 2) == moe.MOE_EINVAL
    assert _mm(wsp=FAKE + 8) == moe.MOE_EINVAL
    assert _mm(aq=1) == moe.MOE_EINVAL and "act_quant" in moe.last_error()
    assert _mm(_w(moe.MOE_I8), aq=2) == moe.MOE_EINVAL
    assert _mm(path=3) == moe.MOE_EINVAL
    assert _mm(path=2) == moe.MOE_EINVAL and "GEMV" in moe.last_error()      # 128 slots
    assert _mm(path=2, T=33) == moe.MOE_EINVAL
    assert _mm(_w(moe.MOE_I8, cols=16400), path=2, T=1) == moe.MOE_EINVAL
    assert _mm(path=-1) == moe.MOE_EINVAL
    assert _mm(T=0) == moe.MOE_OK
    assert _mm(_w(rows=1 << 25), T=1000, rw=FAKE, ws=16) == moe.MOE_ELIMIT and "weighted sum" in moe.last_error()  # more blocks than a dispatch holds
    w = moe.c_moe_weights(moe.MOE_I8, FAKE, None, 8, 64, 128)
    assert _mm(w) == moe.MOE_EINVAL and "scales" in moe.last_error()


def test_path_choice():
    for typ in (moe.MOE_BF16, moe.MOE_F16, moe.MOE_I8):
        assert moe.moe_select_path_typed(1, 4, 32, 2880, typ) == 2
        assert moe.moe_select_path_typed(16, 4, 16, 2880, typ) == 2      # 64 slots, four an expert
        assert moe.moe_select_path_typed(16, 4, 15, 2880, typ) == 1
        assert moe.moe_select_path_typed(17, 4, 32, 2880, typ) == 1
        assert moe.moe_select_path_typed(12, 1, 1, 2880, typ) == 2 and moe.moe_select_path_typed(13, 1, 1, 2880, typ) == 1
        assert moe.moe_select_path_typed(1, 4, 32, 2880, typ, path=1) == 1
    assert moe.moe_select_path_typed(1, 4, 32, 16400, moe.MOE_I8) == 1
    assert moe.moe_select_path_typed(1, 4, 32, 16400, moe.MOE_F16) == 2


def test_fused_ffn_refuses_these_experts():
    for typ in (moe.MOE_BF16, moe.MOE_F16, moe.MOE_I8):
        g, d = _w(typ), _w(typ, rows=128, cols=64)
        r = moe.lib.moe_ffn_fused(ctypes.byref(g), ctypes.byref(g), ctypes.byref(d), None, None, None, FAKE,
                                  moe.MOE_BF16, FAKE, FAKE, 4, 2, FAKE, None, FAKE, 1 << 40, None)
        assert r == moe.MOE_EINVAL and "weight type" in moe.last_error()


def _bw(w=None, st=moe.MOE_BF16, dt=moe.MOE_BF16, path=0, aq=0, ws=1 << 40, x=FAKE, T=64, k=2, B=1, rw=None,
        dx=2 * FAKE, dw=3 * FAKE, dwt=moe.MOE_BF16, dr=None, dy=4 * FAKE, wsp=FAKE):
    opt = moe._options(path, act_quant=aq)
    return moe.lib.moe_mul_mat_id_backward(ctypes.byref(w or _w()), x, st, B, FAKE, T, k, rw, dy, dt, dx, dw, dwt, dr,
                                           ctypes.byref(opt), wsp, ws, None)


def test_gradient_validation():
    assert _bw(ws=16) == moe.MOE_EWORKSPACE
    assert _bw(ws=16, dt=moe.MOE_F32, dwt=moe.MOE_F32, rw=FAKE, dr=FAKE) == moe.MOE_EWORKSPACE
    assert _bw(_w(moe.MOE_I8)) == moe.MOE_EINVAL
    assert _bw(_w(moe.MOE_F32), st=moe.MOE_F32) == moe.MOE_EINVAL
    assert _bw(st=moe.MOE_F16) == moe.MOE_EINVAL
    assert _bw(dt=moe.MOE_F16) == moe.MOE_EINVAL
    assert _bw(dwt=moe.MOE_F16) == moe.MOE_EINVAL
    assert _bw(dx=None, dw=None) == moe.MOE_EINVAL
    assert _bw(dr=FAKE) == moe.MOE_EINVAL and "route_w" in moe.last_error()
    assert _bw(B=3) == moe.MOE_EINVAL
    assert _bw(path=2) == moe.MOE_EINVAL
    assert _bw(aq=1) == moe.MOE_EINVAL
    assert _bw(x=FAKE + 8) == moe.MOE_EINVAL
    assert _bw(dx=2 * FAKE + 8) == moe.MOE_EINVAL
    assert _bw(dw=3 * FAKE + 8) == moe.MOE_EINVAL
    for same in (dict(dx=FAKE), dict(dx=4 * FAKE), dict(dx=FAKE << 4, w=_w(data=FAKE << 4)), dict(dw=FAKE), dict(dw=2 * FAKE), dict(dw=4 * FAKE)):
        assert _bw(**same) == moe.MOE_EINVAL and "inputs" in moe.last_error()
    assert _bw(wsp=FAKE + 8) == moe.MOE_EINVAL
    assert _bw(dy=None) == moe.MOE_EINVAL
    assert _bw(_w(cols=100)) == moe.MOE_ELIMIT
    assert _bw(T=1 << 22) == moe.MOE_ELIMIT
    assert _bw(T=0, dw=None) == moe.MOE_OK
    size = moe.lib.moe_mul_mat_id_backward_workspace_size
    assert size(ctypes.byref(_w()), moe.MOE_BF16, 1, 64, 2, 0, 3, None) > 64 * 2 * 128 * 4
    assert size(ctypes.byref(_w()), moe.MOE_BF16, 1, 64, 2, 0, 4, None) == 0
    assert size(None, moe.MOE_BF16, 1, 64, 2, 0, 3, None) == 0


def test_quantize_rows_validation():
    f = moe.lib.moe_quantize_rows
    assert f(FAKE, moe.MOE_Q8_0, 4, 8, FAKE, FAKE, None) == moe.MOE_EINVAL
    assert f(FAKE, moe.MOE_F16, -1, 8, FAKE, FAKE, None) == moe.MOE_EINVAL
    assert f(FAKE, moe.MOE_F16, 4, 0, FAKE, FAKE, None) == moe.MOE_EINVAL
    assert f(None, moe.MOE_F16, 4, 8, FAKE, FAKE, None) == moe.MOE_EINVAL
    assert f(FAKE + 1, moe.MOE_F16, 4, 8, FAKE, FAKE, None) == moe.MOE_EINVAL
    assert f(FAKE + 2, moe.MOE_F32, 4, 8, FAKE, FAKE, None) == moe.MOE_EINVAL
    assert f(FAKE, moe.MOE_F32, 4, 8, FAKE, FAKE + 2, None) == moe.MOE_EINVAL
    for x, q, d in ((FAKE, FAKE, 2 * FAKE), (FAKE, 2 * FAKE, FAKE), (FAKE, 2 * FAKE, 2 * FAKE)):
        assert f(x, moe.MOE_F32, 4, 8, q, d, None) == moe.MOE_EINVAL and "overlap" in moe.last_error()
    assert f(None, moe.MOE_F32, 0, 8, None, None, None) == moe.MOE_OK


def test_weights_types():
    t = torch.zeros((2, 16, 32))
    assert moe.Weights(t.to(torch.bfloat16)).c().type == moe.MOE_BF16
    assert moe.Weights(t.to(torch.float16)).c().type == moe.MOE_F16
    assert moe.Weights(t).c().type == moe.MOE_F32
    assert moe.Weights(t.to(torch.int8), torch.zeros((2, 16))).c().type == moe.MOE_I8
    with pytest.raises(ValueError):
        moe.Weights(t.to(torch.int8), torch.zeros((2, 15))).c()
    with pytest.raises(ValueError):
        moe.Weights(t.double()).c()
    with pytest.raises(ValueError):
        moe._wanted("src1")
    with pytest.raises(ValueError):
        moe._wanted(("src2",))
