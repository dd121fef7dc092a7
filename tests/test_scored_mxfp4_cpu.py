"""CPU checks for scored routing, its gradient and MXFP4 activations: the float64 forms the GPU
tests compare against are pinned to torch and to differences, and the library refuses bad
arguments before any HIP call."""
import ctypes

import numpy as np
import pytest
import torch

import indirect_expert_matmul_amd as moe
import oracle
import ref64

FAKE = 0x10000  # never dereferenced: every call below fails validation first


def _logits(T, E, seed, spread=2.0):
    return np.random.default_rng(seed).standard_normal((T, E)) * spread


# ---------------------------------------------------------------- the float64 forms
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_matches_torch_topk(score):
    l = _logits(40, 24, 1)
    bias = np.random.default_rng(2).standard_normal(24) * 0.1
    ids, w, s = ref64.route(l, 5, bias=bias, score=score, renorm=False, scale=2.5)
    lt = torch.from_numpy(l)
    st = torch.softmax(lt, 1) if score == "softmax" else torch.sigmoid(lt)
    ti = torch.topk(st + torch.from_numpy(bias), 5).indices
    assert np.array_equal(ids, ti.numpy())
    assert np.allclose(w, 2.5 * st.gather(1, ti).numpy(), rtol=1e-14)
    assert np.allclose(s, st.numpy(), rtol=1e-13)


def test_route_groups_by_hand():
    """Six experts in three groups: group sums pick the second and third group although the
    largest single choice sits in the first."""
    p = np.array([[0.9, 0.0, 0.6, 0.5, 0.55, 0.5]])
    l = np.log(p / (1 - p + 1e-300) + 1e-300)
    ids, w, _ = ref64.route(l, 2, bias=np.zeros(6), score="sigmoid", n_group=3, topk_group=2, group_top=2)
    assert ids.tolist() == [[2, 4]]
    assert np.allclose(w, [[0.6 / 1.15, 0.55 / 1.15]])
    ids, _, _ = ref64.route(l, 2, bias=np.zeros(6), score="sigmoid", n_group=3, topk_group=1, group_top=1)
    assert ids.tolist() == [[0, 1]]


def test_route_softmax_renormalised_is_the_router_topk():
    """Without bias and groups, renormalised softmax scores are the softmax over the picks."""
    l = _logits(30, 33, 3).astype(np.float32)
    ids, w, _ = ref64.route(l, 6)
    rid, rw = oracle.router_topk(l, 6)
    assert np.array_equal(ids, rid)
    assert np.allclose(w, rw, rtol=1e-13)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_matches_autograd_and_differences(score, renorm):
    rng = np.random.default_rng(5)
    T, E, k = 6, 12, 3
    l = _logits(T, E, 4)
    ids, _, _ = ref64.route(l, k, score=score)
    dw, ds = rng.standard_normal((T, k)), rng.standard_normal((T, E))
    got, _ = ref64.route_backward(l, ids, dw, ds, score, renorm, 1.5)

    def loss(lt):
        s = torch.softmax(lt, 1) if score == "softmax" else torch.sigmoid(lt)
        w = s.gather(1, torch.from_numpy(ids).long())
        if renorm:
            w = w / w.sum(1, keepdim=True)
        return (1.5 * w * torch.from_numpy(dw)).sum() + (s * torch.from_numpy(ds)).sum()
    lt = torch.from_numpy(l).requires_grad_(True)
    loss(lt).backward()
    assert np.allclose(got, lt.grad.numpy(), rtol=1e-11, atol=1e-13)
    h = 1e-6
    for t, e in ((0, 0), (2, 7), (5, int(ids[5, 1]))):
        lp, lm = l.copy(), l.copy()
        lp[t, e] += h
        lm[t, e] -= h
        d = (loss(torch.from_numpy(lp)) - loss(torch.from_numpy(lm))).item() / (2 * h)
        assert abs(d - got[t, e]) < 1e-7


def test_quantize_by_hand_and_nearest():
    x = np.zeros((1, 64))
    x[0, :10] = [8.0, -0.5, 0.25, 0.75, 5.0, 7.0, -2.5, 3.0, 1e-9, -1e-9]
    codes, byte = ref64.quantize(x)
    assert byte.tolist() == [[128, 0]]                    # floor(log2 8) - 2 = 1
    # scaled by 2: 4, -.25, .125, .375, 2.5, 3.5, -1.25, 1.5, ~0, ~-0
    assert codes[0, :10].tolist() == [6, 8, 0, 1, 4, 6, 10, 3, 0, 8]
    v = np.linspace(-7.9, 7.9, 4001)
    q = ref64.E2M1[ref64.nearest(v)]
    step = np.where(np.abs(v) < 2, 0.5, np.where(np.abs(v) < 4, 1.0, 2.0))
    assert np.all(np.abs(q - np.clip(v, -6, 6)) <= step / 2 + 1e-12)
    for c in range(16):
        assert oracle.e2m1_to_double(c) == ref64.E2M1[c]
    packed = ref64.pack(codes)
    assert np.array_equal(ref64.unpack(packed), codes)


# ---------------------------------------------------------------- refusals
def test_mxfp4_act_validation():
    def w(typ=moe.MOE_MXFP4, n_mat=8, rows=64, cols=128, data=FAKE):
        return moe.c_moe_weights(typ, data, FAKE, n_mat, rows, cols)

    def mm(wt=None, path=0, ws=1 << 40, x=FAKE, aq=2, T=64, k=2):
        opt = moe._options(path, act_quant=aq)
        return moe.lib.moe_mul_mat_id(ctypes.byref(wt or w()), x, moe.MOE_BF16, 1, FAKE, T, k, None, FAKE,
                                      ctypes.byref(opt), FAKE, ws, None)
    assert mm(ws=16) == moe.MOE_EWORKSPACE                # valid up to the workspace
    assert mm(wt=w(moe.MOE_Q8_0)) == moe.MOE_EINVAL
    assert "MXFP4" in moe.last_error()
    assert mm(wt=w(moe.MOE_IQ4_NL)) == moe.MOE_EINVAL
    assert mm(aq=3) == moe.MOE_EINVAL
    assert mm(aq=-1) == moe.MOE_EINVAL
    assert mm(path=7) == moe.MOE_EINVAL
    assert mm(path=2) == moe.MOE_EINVAL                   # 128 slots: past the GEMV's 64
    assert "GEMV" in moe.last_error()
    assert mm(path=2, T=32, x=FAKE + 2) == moe.MOE_EINVAL
    assert mm(path=2, T=32, wt=w(data=FAKE + 8)) == moe.MOE_EINVAL
    assert mm(path=2, T=1, wt=w(cols=100)) == moe.MOE_ELIMIT
    assert mm(x=FAKE + 2) == moe.MOE_EINVAL               # activations not 16-byte aligned
    assert mm(wt=w(data=FAKE + 8)) == moe.MOE_EINVAL      # codes not 16-byte aligned
    assert mm(wt=w(cols=100)) == moe.MOE_ELIMIT
    assert mm(T=0) == moe.MOE_OK
    opt = moe._options(0, act_quant=2)
    g, d = w(), w(rows=128, cols=64)
    def ffn(g=g, d=d, ws=16):
        return moe.lib.moe_ffn_fused(ctypes.byref(g), ctypes.byref(g), ctypes.byref(d), None, None, None, FAKE,
                                     moe.MOE_BF16, FAKE, FAKE, 16, 2, FAKE, ctypes.byref(opt), FAKE, ws, None)
    assert ffn() == moe.MOE_EWORKSPACE                    # the GEMV path's h
    assert ffn(g=w(moe.MOE_Q8_0), d=w(moe.MOE_Q8_0, rows=128, cols=64)) == moe.MOE_EINVAL
    assert ffn(d=w(rows=128, cols=64, data=FAKE + 4), ws=1 << 40) == moe.MOE_EINVAL
    assert moe.lib.moe_ffn_fused_workspace_size(ctypes.byref(g), None, moe.MOE_BF16, 16, 2, ctypes.byref(opt)) > 0
    typed = moe.moe_select_path_typed
    assert typed(4096, 4, 32, 2880, moe.MOE_MXFP4, act_quant=2) == 4
    assert typed(1, 4, 32, 2880, moe.MOE_MXFP4, act_quant=2) == 5
    assert typed(1, 4, 32, 2880, moe.MOE_MXFP4, path=moe.PATH_GEMM, act_quant=2) == 4
    assert typed(16, 4, 32, 2880, moe.MOE_MXFP4, path=moe.PATH_GEMV, act_quant=2) == 5
    for typ in (moe.MOE_Q8_0, moe.MOE_IQ4_XS):
        with pytest.raises(moe.MoeError):
            moe.moe_select_path_typed(4, 4, 32, 2880, typ, act_quant=2)


def test_mxfp4_act_path_bounds():
    def typed(T, k, width, path=moe.PATH_AUTO):
        return moe.moe_select_path_typed(T, k, 32, width, moe.MOE_MXFP4, path=path, act_quant=2)
    assert [typed(T, k, 128) for T, k in ((64, 1), (16, 4), (1, 64), (65, 1), (13, 5))] == [5, 5, 5, 4, 4]
    def few(T, path=moe.PATH_AUTO):
        return moe.moe_select_path_typed(T, 1, 2, 128, moe.MOE_MXFP4, path=path, act_quant=2)
    assert few(32) == 5 and few(33) == 4 and few(33, moe.PATH_GEMV) == 5    # 16 slots an expert on average
    assert typed(1, 1, 127) == 4 and typed(1, 1, 96) == 4
    for T, k, width in ((1, 1, 96), (65, 1, 128)):
        with pytest.raises(moe.MoeError):
            typed(T, k, width, path=moe.PATH_GEMV)


def test_quantize_mxfp4_validation():
    q = moe.lib.moe_quantize_mxfp4
    assert q(FAKE, moe.MOE_BF16, 4, 100, FAKE, FAKE, None, None) == moe.MOE_ELIMIT
    assert q(FAKE, moe.MOE_Q8_0, 4, 64, FAKE, FAKE, None, None) == moe.MOE_EINVAL
    assert q(FAKE, moe.MOE_BF16, -1, 64, FAKE, FAKE, None, None) == moe.MOE_EINVAL
    assert q(None, moe.MOE_BF16, 4, 64, FAKE, FAKE, None, None) == moe.MOE_EINVAL
    assert q(FAKE + 4, moe.MOE_F32, 4, 64, FAKE, FAKE, None, None) == moe.MOE_EINVAL
    assert q(FAKE, moe.MOE_F32, 4, 64, FAKE, FAKE, FAKE + 2, None) == moe.MOE_EINVAL
    assert q(FAKE, moe.MOE_F32, 1 << 31, 32, FAKE, FAKE, None, None) == moe.MOE_ELIMIT
    assert q(FAKE, moe.MOE_F32, 1 << 62, 1 << 20, FAKE, FAKE, None, None) == moe.MOE_ELIMIT
    assert q(None, moe.MOE_BF16, 0, 64, None, None, None, None) == moe.MOE_OK
    with pytest.raises(ValueError):
        moe.moe_quantize_mxfp4(torch.zeros((4, 33)))
    with pytest.raises(ValueError):
        moe.moe_quantize_mxfp4(torch.zeros((4, 64)))      # not on the GPU


def test_router_scored_validation():
    def call(T=4, E=64, k=4, dt=moe.MOE_F32, score=0, G=1, keep=1, top=2, renorm=1, scale=1.0, lg=FAKE, cfg=True,
             scores=None):
        c = moe.c_moe_router_config(score, G, keep, top, renorm, scale)
        return moe.lib.moe_router_scored(lg, dt, None, T, E, k, ctypes.byref(c) if cfg else None, FAKE, FAKE,
                                         scores, None)
    assert call(T=0) == moe.MOE_OK
    assert call(dt=moe.MOE_Q8_0) == moe.MOE_EINVAL
    assert call(cfg=False) == moe.MOE_EINVAL
    assert call(lg=None) == moe.MOE_EINVAL
    assert call(scores=FAKE) == moe.MOE_EINVAL            # in the place of logits
    assert call(k=0) == moe.MOE_EINVAL
    assert call(k=65) == moe.MOE_EINVAL
    assert call(E=1025) == moe.MOE_ELIMIT
    assert call(T=1 << 22) == moe.MOE_ELIMIT
    assert call(score=2) == moe.MOE_EINVAL
    assert call(G=5) == moe.MOE_EINVAL                    # does not divide 64
    assert call(G=0) == moe.MOE_EINVAL
    assert call(G=8, keep=9) == moe.MOE_EINVAL
    assert call(G=8, keep=0) == moe.MOE_EINVAL
    assert call(G=8, keep=2, k=17) == moe.MOE_EINVAL      # two groups of eight hold 16
    assert "kept groups" in moe.last_error()
    assert call(top=3) == moe.MOE_EINVAL
    assert call(renorm=2) == moe.MOE_EINVAL
    assert call(scale=float("nan")) == moe.MOE_EINVAL
    assert call(scale=float("inf")) == moe.MOE_EINVAL
    for bad in (torch.zeros(4, 8), torch.zeros(4, 8, dtype=torch.float16), torch.zeros(8)):
        with pytest.raises(ValueError):
            moe.moe_router_scored(bad, 2)                 # host tensor, float16, one dimension


def test_router_scored_backward_validation():
    def call(T=4, E=64, k=4, dt=moe.MOE_F32, ds=None, stride=0, ids=FAKE, score=1):
        c = moe.c_moe_router_config(score, 0, 0, 0, 1, 1.0)   # group fields are not read
        return moe.lib.moe_router_scored_backward(FAKE, dt, ids, FAKE, ds, stride, T, E, k, ctypes.byref(c),
                                                  FAKE, None)
    assert call(T=0) == moe.MOE_OK
    assert call(dt=moe.MOE_MXFP4) == moe.MOE_EINVAL
    assert call(ids=None) == moe.MOE_EINVAL
    assert call(ds=FAKE, stride=63) == moe.MOE_EINVAL
    assert call(ds=FAKE, stride=-64) == moe.MOE_EINVAL
    assert call(score=-1) == moe.MOE_EINVAL
    assert call(E=0) == moe.MOE_EINVAL
    assert call(k=1024) == moe.MOE_ELIMIT
