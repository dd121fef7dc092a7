"""GPU parity of moe_router_scored and moe_router_scored_backward against the float64 forms of
ref64: ids equal, weights, scores and gradients within the rounding bounds ref64 derives (a
bfloat16 gradient adds half a step, 2^-8 of the value)."""
import numpy as np
import pytest
import torch

import indirect_expert_matmul_amd as moe
import ref64
import synth
from moe_testutil import dev_f32, dev_i32, run_ffn, upload_ffn

pytestmark = pytest.mark.gpu


def _logits(T, E, seed, dtype=torch.float32, spread=1.5):
    """(device logits, their float64 values)."""
    l = torch.from_numpy(np.random.default_rng(seed).standard_normal((T, E)) * spread).to(dtype)
    return l.cuda(), l.double().numpy()


def _check_route(dev, l, k, bias=None, **kw):
    got = moe.moe_router_scored(dev, k, bias=None if bias is None else dev_f32(bias), return_scores=True, **kw)
    plain = moe.moe_router_scored(dev, k, bias=None if bias is None else dev_f32(bias), **kw)
    torch.cuda.synchronize()
    assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])   # with and without the scores
    ids, w, s = ref64.route(l, k, bias=None if bias is None else np.float32(bias), **kw)
    gi, gw, gs = (t.cpu().numpy() for t in got)
    assert np.array_equal(gi, ids)
    for t in range(l.shape[0]):
        rel = ref64.rounding(l[t], l.shape[1] + k)
        assert np.all(np.abs(gw[t] - w[t]) <= rel * np.abs(w[t]) + 1e-38), t
        assert np.all(np.abs(gs[t] - s[t]) <= rel * s[t] + 1e-38), t
    return gi, gw, gs


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,G,keep,top,score,renorm,scale,bias", [
    (1, 256, 8, 8, 4, 2, "sigmoid", True, 2.5, True),       # one token, grouped
    (67, 256, 8, 8, 4, 2, "sigmoid", True, 2.5, True),
    (130, 64, 6, 1, 1, 2, "softmax", False, 1.0, False),
    (33, 128, 8, 1, 1, 1, "softmax", True, 1.0, False),
    (50, 160, 6, 8, 3, 1, "softmax", False, 16.0, False),   # group maxima, no bias
    (50, 160, 6, 8, 3, 2, "softmax", True, 1.0, False),     # group sums of scores, no bias
    (9, 7, 7, 7, 7, 2, "sigmoid", False, -1.0, True),       # groups of one, all kept
    (11, 12, 3, 4, 2, 2, "softmax", True, 1.0, True),
    (5, 1, 1, 1, 1, 1, "sigmoid", True, 1.0, False),        # one expert
    (6, 1024, 32, 32, 5, 2, "sigmoid", True, 1.0, True),
    (3, 1000, 999, 1, 1, 1, "softmax", True, 1.0, True),
    (4, 1024, 512, 512, 256, 1, "sigmoid", True, 1.0, False),   # many small groups
    (19, 96, 24, 3, 1, 2, "softmax", True, 1.0, True),      # picks fill most of one group
])
def test_route_parity(T, E, k, G, keep, top, score, renorm, scale, bias, dtype):
    dev, l = _logits(T, E, T + E, dtype)
    b = np.random.default_rng(E).standard_normal(E) * 0.05 if bias else None
    _check_route(dev, l, k, bias=b, n_group=G, topk_group=keep, group_top=top, score=score, renorm=renorm, scale=scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_config_shapes(score):
    for name in ("lite", "dec8", "skew"):
        cfg = synth.CONFIGS[name]
        T = min(cfg.n_tokens, 300)
        lg = synth.draw_router_logits(cfg.seed, T, cfg.n_experts)
        _check_route(dev_f32(lg), lg.astype(np.float64), cfg.n_used, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_route_ties_take_the_lower_index(score, bias):
    """Few distinct logits: equal choices, equal groups, and choices that differ only past float32."""
    rng = np.random.default_rng(3)
    l = rng.integers(-2, 3, size=(64, 64)).astype(np.float64)
    b = rng.integers(0, 2, size=64) * 0.25 if bias else None
    for G, keep, top in ((1, 1, 1), (8, 3, 1), (8, 3, 2)):
        _check_route(dev_f32(l), l, 9, bias=b, score=score, n_group=G, topk_group=keep, group_top=top)
    near = np.float32(1.0) + np.float32(2.0 ** -23) * rng.integers(0, 3, size=(64, 64)).astype(np.float32)
    _check_route(dev_f32(near), near.astype(np.float64), 9, bias=b, score=score)
    _check_route(dev_f32(near), near.astype(np.float64), 9, bias=b, score=score, n_group=4, topk_group=2)
    if bias:   # sums next to each other: score and bias trade places
        s = 1 / (1 + np.exp(-near.astype(np.float64)))
        b2 = (0.9 - s[0]).astype(np.float32)
        _check_route(dev_f32(near), near.astype(np.float64), 9, bias=b2, score="sigmoid")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("big", [2.0 ** 12, 2.0 ** 20, 1e30])
def test_group_sums_that_cancel(score, big):
    """Large balance biases of both signs: a group's two choices cancel, and the groups' order hangs
    on what float32 sums have lost. (1e30: on nothing but the group index.)"""
    T, E, G = 256, 64, 8
    dev, l = _logits(T, E, 4, spread=2.0)
    b = np.full(E, -big)
    b[::E // G] = big
    for keep in (1, 3):
        _check_route(dev, l, keep, bias=b, score=score, n_group=G, topk_group=keep)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_masks_and_extremes(score):
    nan, inf, low = np.nan, np.inf, np.finfo(np.float32).min
    E = 70
    _, l = _logits(12, E, 8)
    l = l.astype(np.float32).astype(np.float64)
    l[0, :] = -inf                       # nothing left: every pick -1
    l[1, :] = nan
    l[2, 3:] = -inf                      # three experts left for six picks
    l[3, ::2] = nan
    l[4, 5], l[4, 66] = inf, inf
    l[5, :] = low                        # a mask of the lowest value is a number
    l[6, :] = low
    l[6, 9] = 0.0
    l[7, :35] = -inf                     # the first groups empty
    l[8, :] = -200.0                     # scores that underflow, weights that do not
    l[8, 4] = -199.0
    l[9, :] = 60.0                       # sigmoids that round to 1
    l[9, 7] = 61.0
    l[10, 0], l[10, 1] = -0.0, 0.0
    for kw in (dict(), dict(n_group=10, topk_group=2), dict(n_group=10, topk_group=2, group_top=1),
               dict(renorm=False)):
        gi, gw, _ = _check_route(dev_f32(l), l, 6, score=score, **kw)
        assert np.all(gi[:2] == -1) and np.all(gw[:2] == 0)
        assert np.all(gi[2, 3:] == -1) and np.all(gi[2, :3] >= 0)
    b = np.random.default_rng(1).standard_normal(E) * 0.1
    b[4], b[11], b[20] = -inf, nan, inf
    gi, _, _ = _check_route(dev_f32(l), l, 6, bias=b, score=score)
    assert not np.isin(gi, (4, 11)).any() and gi[11, 0] == 20


def test_route_out_arguments_stream_and_repeats():
    dev, l = _logits(2000, 256, 5)
    b = dev_f32(np.random.default_rng(2).standard_normal(256) * 0.05)
    kw = dict(bias=b, score="sigmoid", n_group=8, topk_group=4, scale=2.5)
    ref = moe.moe_router_scored(dev, 8, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        ids = torch.full((2000, 8), -7, dtype=torch.int32, device="cuda")
        w = torch.full((2000, 8), np.nan, device="cuda")
        torch.cuda.synchronize()
        got = moe.moe_router_scored(dev, 8, ids=ids, route_w=w, stream=side, **kw)
        side.synchronize()
        assert got[0] is ids and torch.equal(ids, ref[0]) and torch.equal(w, ref[1])
    e = moe.moe_router_scored(torch.zeros((0, 16), device="cuda"), 4)
    assert e[0].shape == (0, 4)
    with pytest.raises(ValueError):
        moe.moe_router_scored(dev, 8, bias=b[:255])
    with pytest.raises(ValueError):
        moe.moe_router_scored(dev.t(), 8)
    with pytest.raises(ValueError):
        moe.moe_router_scored(dev, 8, score="tanh")
    with pytest.raises(moe.MoeError):
        moe.moe_router_scored(dev, 257)


# ---------------------------------------------------------------- gradient
def _check_grad(dev, l, ids, seed, aux, score, renorm, scale):
    rng = np.random.default_rng(seed)
    T, E = l.shape
    dw = rng.standard_normal(ids.shape).astype(np.float32)
    ds = {"none": None, "row": rng.standard_normal(E), "full": rng.standard_normal((T, E))}[aux]
    ds = None if ds is None else ds.astype(np.float32)
    got = moe.moe_router_scored_backward(dev, dev_i32(ids), dev_f32(dw), d_scores=None if ds is None else dev_f32(ds),
                                         score=score, renorm=renorm, scale=scale)
    torch.cuda.synchronize()
    assert got.dtype == dev.dtype
    ref, bound = ref64.route_backward(l, ids, dw, ds, score, renorm, scale)
    if dev.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (np.abs(ref) + bound)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= bound + 1e-37), (err - bound).max()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,aux", [(1, 256, 8, "none"), (37, 160, 6, "row"), (66, 64, 6, "full"),
                                       (9, 33, 33, "full"), (5, 1024, 100, "row"), (4, 1, 1, "full")])
def test_grad_parity(T, E, k, aux, score, renorm, dtype):
    dev, l = _logits(T, E, T * 7 + E, dtype)
    ids, _, _ = ref64.route(l, k, score=score)
    _check_grad(dev, l, ids, T, aux, score, renorm, 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_grad_masks_invalid_and_repeated_ids(score, renorm):
    E = 70
    _, l = _logits(9, E, 21)
    l = l.astype(np.float32).astype(np.float64)
    rng = np.random.default_rng(4)
    ids = np.stack([rng.permutation(E)[:5] for _ in range(9)]).astype(np.int32)
    l[0, :] = -np.inf
    l[1, ::3] = np.nan
    l[2, ids[2, 1]] = -np.inf            # a pick whose logit is masked
    ids[3, 2], ids[3, 4] = -1, E + 3
    ids[4] = ids[4, 0]                   # the same expert five times
    ids[5, 3] = ids[5, 1]
    ids[6] = -1
    l[7, :] = -200.0
    l[8, :] = 40.0
    for aux in ("none", "full"):
        _check_grad(dev_f32(l), l, ids, 3, aux, score, renorm, 1.0)


def test_grad_in_place_strides_and_repeats():
    dev, l = _logits(500, 96, 2)
    ids, _ = moe.moe_router_scored(dev, 4, score="sigmoid")
    dw = torch.randn((500, 4), device="cuda")
    wide = torch.randn((500, 128), device="cuda")          # rows 128 apart through the C call
    c = moe._router_config("sigmoid", 1, 1, 1, True, 1.0)
    ref = moe.moe_router_scored_backward(dev, ids, dw, d_scores=wide[:, :96].contiguous(), score="sigmoid")
    out = torch.empty_like(dev)
    st = moe.lib.moe_router_scored_backward(dev.data_ptr(), moe.MOE_F32, ids.data_ptr(), dw.data_ptr(),
                                            wide.data_ptr(), 128, 500, 96, 4, moe.ctypes.byref(c), out.data_ptr(),
                                            torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == moe.MOE_OK and torch.equal(out, ref)
    buf = dev.clone()
    moe.moe_router_scored_backward(buf, ids, dw, d_scores=wide[:, :96].contiguous(), score="sigmoid", out=buf)
    torch.cuda.synchronize()
    assert torch.equal(buf, ref)
    with pytest.raises(ValueError):
        moe.moe_router_scored_backward(dev, ids, dw[:, :3], score="sigmoid")
    with pytest.raises(ValueError):
        moe.moe_router_scored_backward(dev, ids, dw, d_scores=wide, score="sigmoid")


def test_forward_and_gradient_as_a_training_step_uses_them():
    """Gradient against differences of the forward call itself (float64 of its float32 outputs): the
    step is large against float32 rounding and the picks stay the same ones."""
    T, E, k = 8, 32, 4
    dev, l = _logits(T, E, 31)
    kw = dict(score="sigmoid", renorm=True, scale=2.5)
    ids, w = moe.moe_router_scored(dev, k, **kw)
    dw = torch.randn((T, k), device="cuda")
    grad = moe.moe_router_scored_backward(dev, ids, dw, **kw).double().cpu()
    h = 2.0 ** -8
    for e in (0, 5, 31, int(ids[0, 0]), int(ids[3, 2])):
        up, dn = dev.clone(), dev.clone()
        up[:, e] += h
        dn[:, e] -= h
        iu, wu = moe.moe_router_scored(up, k, **kw)
        il, wl = moe.moe_router_scored(dn, k, **kw)
        same = ((iu == ids).all(1) & (il == ids).all(1)).cpu()
        d = (((wu - wl).double() * dw.double()).sum(1) / (2 * h)).cpu()
        # |third derivative| h^2 / 6 and the rounding of 2.5 * k weights over 2 h
        tol = 2.5 * dw.abs().sum(1).cpu() * (h * h + 16 * ref64.EPS / h)
        assert ((d - grad[:, e]).abs() <= tol)[same].all()
        assert same.float().mean() > 0.5


def test_router_feeds_layer_and_graph_replays():
    """Masked (padding) tokens, grouped routing and the layer behind it, eager and captured."""
    E, k, T = 16, 4, 40
    inp = synth.make_custom_ffn(5, E, k, T, 128, 96, 1)
    dv = upload_ffn(inp)
    dev, _ = _logits(T, E, 6)
    dev[7] = -float("inf")
    kw = dict(score="sigmoid", n_group=4, topk_group=2, scale=2.5)
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    rw = torch.empty((T, k), device="cuda")
    out = torch.empty((T, 128), device="cuda")
    grad = torch.empty_like(dev)
    dw = torch.randn((T, k), device="cuda")
    ws = torch.empty(moe.moe_ffn_fused_workspace_size(dv["gate"], dv["shared"][0], T, k), dtype=torch.uint8,
                     device="cuda")

    def layer():
        moe.moe_router_scored(dev, k, ids=ids, route_w=rw, **kw)
        dv["ids"], dv["route_w"] = ids, rw
        run_ffn(dv, out=out, workspace=ws)
        moe.moe_router_scored_backward(dev, ids, dw, score="sigmoid", scale=2.5, out=grad)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.synchronize()
    ref = [t.clone() for t in (ids, rw, out, grad)]
    assert (ids[7] == -1).all() and (rw[7] == 0).all() and (grad[7] == 0).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer()
    for _ in range(4):
        for t in (rw, out, grad):
            t.fill_(float("nan"))
        ids.fill_(-5)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((ids, rw, out, grad), ref))
        torch.randn(1 << 18, device="cuda").sum().item()
