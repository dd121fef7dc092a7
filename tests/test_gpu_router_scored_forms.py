"""GPU checks of scored routing and its gradient at the edges of their number formats, against the
float64 forms of ref64."""
import numpy as np
import pytest
import torch

import indirect_expert_matmul_amd as moe
import ref64
from moe_testutil import dev_f32, dev_i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_group_sums_past_float32(score, dtype):
    """Biases of the lowest float32 as a mask: the sum of two of them is no float32, but it ranks its
    group above groups without an expert, and sums past the range above 0 rank by their size."""
    low = np.finfo(np.float32).min
    l = torch.from_numpy(np.random.default_rng(1).standard_normal((37, 16))).to(dtype)
    b = np.full(16, -np.inf)                 # groups of 4
    b[4:8] = low
    b[8:12] = np.linspace(-0.1, 0.1, 4)
    up = np.zeros(16)
    up[0:4], up[4:8], up[12:16] = -low / 1.5, -low / 1.25, -low
    down = np.array([low / 1.25] * 4 + [low] * 4 + [low / 1.5] * 4 + [low / 1.75] * 4)
    for bias, keep, k in ((b, 2, 6), (b, 3, 9), (up, 1, 3), (up, 2, 7), (down, 1, 2), (down, 3, 12)):
        kw = dict(score=score, n_group=4, topk_group=keep)
        ids, w = moe.moe_router_scored(l.cuda(), k, bias=dev_f32(bias), **kw)
        ri, _, _ = ref64.route(l.double().numpy(), k, bias=np.float32(bias), **kw)
        assert np.array_equal(ids.cpu().numpy(), ri), (keep, k)


def _whole_logits(T, E, lo, hi):
    """Whole numbers: differences of them are exact, so that no bound has a term for their rounding."""
    l = np.random.default_rng(T + E).integers(lo, hi + 1, size=(T, E)).astype(np.float64)
    l[:, :2] = lo, hi
    return l


def _lane(E):
    """Experts of a lane in the kernels of 16 lanes a token: the length of its sum."""
    return next(c for c in (4, 8, 16, 32, 64) if 16 * c >= E)


@pytest.mark.parametrize("E", [40, 128, 160, 512, 600])
def test_scores_to_the_last_bits(E):
    """Roundings of the formulas, an exponential counted as two (1 ulp) at any size of its argument.
    Sigmoid z / (1 + z): 2 + 1 + 1. Softmax: 2 for the numerator, 2 and its additions (one fewer than a
    lane's experts, 4 across the lanes) for the sum, 2 for the quotient."""
    T, k = 50, 5
    for score, l in (("sigmoid", _whole_logits(T, E, -80, 80)), ("softmax", _whole_logits(T, E, -85, 0))):
        n = 4 if score == "sigmoid" else 2 + 2 + _lane(E) + 3 + 2
        tol = n * (1 + 1e-5) * ref64.EPS
        ri, rw, rs = ref64.route(l, k, score=score, renorm=False)
        for bias in (None, dev_f32(np.zeros(E))):
            ids, w, s = moe.moe_router_scored(dev_f32(l), k, bias=bias, score=score, renorm=False, return_scores=True)
            ids2, w2 = moe.moe_router_scored(dev_f32(l), k, bias=bias, score=score, renorm=False)
            assert torch.equal(ids, ids2) and torch.equal(w, w2)
            err = np.abs(s.double().cpu().numpy() - rs) / rs
            assert err.max() <= tol, (score, err.max() / ref64.EPS, n)
            werr = np.abs(w.double().cpu().numpy() - rw) / rw
            assert werr.max() <= tol, (score, werr.max() / ref64.EPS, n)


@pytest.mark.parametrize("E", [40, 128, 160, 512, 600])
def test_score_gradient_to_the_last_bits(E):
    """The gradient through the scores alone. Sigmoid d s (1 - s): one of s and 1 - s is 1 / (1 + z) with
    3 roundings, the other z / (1 + z) with 4 or, as a product, 5; 2 for the products. Softmax
    s d - s sum(s d): n for s as above, 1 for s d, n + 1 and the sum's additions for the sum, 1 each for
    the product and the difference."""
    T = 50
    ids = dev_i32(np.full((T, 2), -1))
    dw = torch.ones((T, 2), device="cuda")
    d = np.random.default_rng(E).uniform(0.5, 2, size=(T, E)).astype(np.float32)
    d[:, ::3] *= -1
    adds = _lane(E) + 3
    n = 2 + 2 + adds + 2
    for score, l in (("sigmoid", _whole_logits(T, E, -80, 80)), ("softmax", _whole_logits(T, E, -85, 0))):
        got = moe.moe_router_scored_backward(dev_f32(l), ids, dw, d_scores=dev_f32(d), score=score)
        s = ref64.scores(l, score)
        d64 = d.astype(np.float64)
        if score == "sigmoid":
            ref = s / (1 + np.exp(l)) * d64
            bound = 10 * np.abs(ref)
        else:
            q = s * d64
            mag = np.abs(q).sum(axis=1, keepdims=True)
            ref = q - s * q.sum(axis=1, keepdims=True)
            bound = (n + 2) * np.abs(q) + (n + (n + 1 + adds) + 2) * s * mag
        err = np.abs(got.double().cpu().numpy() - ref)
        worst = (err / (bound * ref64.EPS)).max()
        assert worst <= 1 + 1e-5, (score, worst)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(40, 5), (256, 8), (512, 15)])
def test_scores_do_not_depend_on_the_bias(E, k, score):
    """Tokens whose choices are too near each other are routed again in float64; their scores stay those of
    the same logits without a bias, bit for bit, infinite logits among them."""
    T = 45
    l = np.random.default_rng(E).integers(-3, 3, size=(T, E)).astype(np.float64) / 7     # many ties
    l = l.astype(np.float32).astype(np.float64)
    l[0], l[1] = 0.3, -np.inf
    l[2, 5], l[3, :3] = np.inf, np.inf
    l[4, ::2] = np.nan
    dev = dev_f32(l)
    plain = moe.moe_router_scored(dev, k, score=score, return_scores=True)
    zero = moe.moe_router_scored(dev, k, bias=torch.zeros(E, device="cuda"), score=score, return_scores=True)
    small = moe.moe_router_scored(dev, k, bias=dev_f32(np.random.default_rng(1).standard_normal(E) * 1e-7), score=score,
                                  return_scores=True)
    for got in (zero, small):
        assert torch.equal(got[2].view(torch.int32), plain[2].view(torch.int32))
    assert np.array_equal(zero[0].cpu().numpy(), ref64.route(l, k, bias=np.zeros(E), score=score)[0])
