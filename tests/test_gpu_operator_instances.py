"""Every size class of the scored routing kernels, tensors that start off their vector alignment, and the
MXFP4 GEMV with several groups of rows a thread block, against the float64 forms of ref64."""
import numpy as np
import pytest
import torch

import indirect_expert_matmul_amd as moe
import ref64
from moe_testutil import dev_f32, dev_i32
from test_gpu_mxfp4_act import _act, _check, _experts, _ffn_case, _mul_mat_id
from test_gpu_router_scored import _check_grad, _check_route, _logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,G,keep,top,bias", [
    (33, 100, 12, 1, 1, 1, True),
    (33, 100, 15, 5, 2, 2, False),
    (21, 256, 12, 8, 3, 2, True),
    (21, 256, 15, 1, 1, 1, True),
    (22, 260, 8, 1, 1, 1, True),
    (22, 260, 15, 4, 2, 2, True),
    (18, 384, 8, 16, 5, 2, True),
    (18, 384, 15, 1, 1, 1, False),
    (17, 512, 8, 8, 4, 1, True),
    (17, 512, 15, 16, 1, 2, True),           # one group of 32 experts
    (13, 512, 16, 16, 1, 2, True),           # past the picks of 16 lanes a token
    (9, 511, 9, 7, 3, 2, True),              # rows that start anywhere
    (5, 1024, 9, 1024, 700, 1, True),        # as many groups as experts
    (19, 16, 5, 16, 5, 2, True),
    (19, 16, 3, 16, 9, 2, False),
    (19, 30, 7, 15, 4, 2, False),            # groups of two
])
def test_route_instances(T, E, k, G, keep, top, bias, score, dtype):
    dev, l = _logits(T, E, T + E + k, dtype)
    b = np.random.default_rng(E + k).standard_normal(E) * 0.05 if bias else None
    for renorm in (True, False):
        _check_route(dev, l, k, bias=b, n_group=G, topk_group=keep, group_top=top, score=score, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(100, 15), (256, 15), (300, 8), (512, 15)])
def test_route_instances_with_few_in_one_lane(E, k, score):
    """All picks in one lane's experts (chunks of 4 every 64), in rising and falling order."""
    l = np.random.default_rng(k).uniform(-1, 0, size=(8, E))
    first = [c + i for c in range(0, E, 64) for i in range(4)]
    for t in range(8):
        v = np.linspace(1, 3, len(first))
        l[t, [e for e in first]] = v if t % 2 else v[::-1]
        l[t] = np.roll(l[t], 4 * t)
    l = l.astype(np.float32).astype(np.float64)
    for b in (None, np.zeros(E), np.linspace(0, 0.01, E)):
        _check_route(dev_f32(l), l, k, bias=b, score=score)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,aux", [(14, 300, 6, "full"), (14, 300, 16, "row"), (9, 512, 16, "none"), (9, 512, 6, "full"),
                                       (11, 64, 20, "full"), (11, 100, 20, "row"), (11, 200, 20, "full"),
                                       (11, 400, 20, "none"), (7, 700, 3, "full")])
def test_grad_instances(T, E, k, aux, score, renorm, dtype):
    dev, l = _logits(T, E, T * 3 + E, dtype)
    ids, _, _ = ref64.route(l, k, score=score)
    ids[1, 0], ids[2, 1] = -1, ids[2, 0]
    _check_grad(dev, l, ids, T, aux, score, renorm, 2.5)


def _off(t, by=1):
    """The same contiguous tensor, starting `by` elements into its storage."""
    buf = torch.empty(t.numel() + by + 8, dtype=t.dtype, device=t.device)
    v = buf[by:by + t.numel()].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(64, 6), (256, 8), (512, 8), (1024, 20)])
def test_tensors_off_their_vector_alignment(E, k, dtype):
    T = 19
    dev, l = _logits(T, E, E + k, dtype)
    b = dev_f32(np.random.default_rng(E).standard_normal(E) * 0.05)
    kw = dict(score="sigmoid", n_group=8, topk_group=4, scale=2.5)
    ids, w, s = moe.moe_router_scored(dev, k, bias=b, return_scores=True, **kw)
    assert dev.data_ptr() % 16 == 0 and _off(dev).data_ptr() % 8 != 0 and _off(b).data_ptr() % 16 != 0
    ri, rw, rs = ref64.route(l, k, bias=b.cpu().numpy(), **kw)
    assert np.array_equal(ids.cpu().numpy(), ri)
    rel = ref64.rounding(l, E + k)
    near = lambda t, ref: np.all(np.abs(t.double().cpu().numpy() - ref) <= rel * np.abs(ref) + 1e-38)
    blank = lambda t: _off(torch.full_like(t, -7))
    for lg, bb, si in ((_off(dev), b, s), (dev, _off(b), s), (dev, b, blank(s)), (_off(dev), _off(b), blank(s))):
        i2, w2, s2 = moe.moe_router_scored(lg, k, bias=bb, ids=blank(ids), route_w=blank(w),
                                           scores=si if si is not s else torch.full_like(s, -7), **kw)
        assert torch.equal(i2, ids) and near(w2, rw) and near(s2, rs)
    dw, ds = torch.randn((T, k), device="cuda"), torch.randn((T, E), device="cuda")
    for score in ("softmax", "sigmoid"):
        for lg, d, o in ((_off(dev), ds, dev), (dev, _off(ds), dev), (dev, ds, _off(dev)), (_off(dev), _off(ds), _off(dev))):
            out = o.clone() if o is dev else o
            out.fill_(7)
            got = moe.moe_router_scored_backward(lg, _off(ids), _off(dw), d, score=score, scale=2.5, out=out)
            ref, bound = ref64.route_backward(l, ri, dw.cpu().numpy(), ds.cpu().numpy(), score, True, 2.5)
            if dtype == torch.bfloat16:
                bound = bound + 2.0 ** -8 * (np.abs(ref) + bound)
            assert np.all(np.abs(got.double().cpu().numpy() - ref) <= bound + 1e-37)


# ---------------------------------------------------------------- MXFP4 GEMV
def _spread(T, k, E, seed):
    """As many distinct experts as there are slots, some slots without one."""
    ids = np.random.default_rng(seed).permutation(E)[:T * k].reshape(T, k).astype(np.int32)
    ids[0, 0], ids[T // 2, k - 1] = -1, E
    return ids


# A block takes 32 rows while experts x column parts x blocks of 32 rows reach 2048, and 64 likewise.
@pytest.mark.parametrize("E,k,T,K,N,B_is_k", [
    (64, 2, 32, 1056, 490, False),    # 32 rows a block; 10 in the last one
    (64, 4, 16, 1056, 506, True),     # 26
    (64, 2, 32, 1056, 1034, False),   # 64 rows a block; 10 in the last one
    (64, 8, 8, 1056, 1050, True),     # 26
    (64, 1, 64, 544, 2096, False),    # 48, one column part
    (40, 5, 8, 2080, 1137, True),     # odd rows, three column parts
])
def test_gemv_with_several_row_groups(E, k, T, K, N, B_is_k):
    _mul_mat_id(E, k, T, K, N, k if B_is_k else 1, _spread(T, k, max(E, T * k), T + N) % (E + 1), moe.PATH_GEMV)


def test_gemv_with_several_row_groups_and_passes():
    """More slots of one expert than a pass takes."""
    rng = np.random.default_rng(3)
    ids = rng.integers(0, 64, size=(32, 2)).astype(np.int32)
    ids[:20] = 5
    _mul_mat_id(64, 2, 32, 1056, 1034, 1, ids, moe.PATH_GEMV)


@pytest.mark.parametrize("E,k,T,n_embd,n_ff,S", [
    (64, 2, 32, 1056, 1056, 0),       # gate/up and down of 64 rows a block, half of the last one's
    (64, 4, 16, 1056, 512, 2),        # gate/up of 32 rows a block
    (16, 1, 16, 7712, 992, 0),        # eight column parts need more LDS than there is: seven
])
def test_ffn_gemv_with_several_row_groups(E, k, T, n_embd, n_ff, S):
    _ffn_case(E, k, T, n_embd, n_ff, S, _spread(T, k, max(E, T * k), n_ff) % (E + 1), path=moe.PATH_GEMV)


@pytest.mark.parametrize("path", [moe.PATH_GEMV, moe.PATH_GEMM])
@pytest.mark.parametrize("T,n_embd,n_ff,n_ff_sh,S", [
    (7, 256, 128, 1184, 2),           # shared experts wider than the routed ones: parts of the columns are theirs alone
    (7, 256, 1184, 128, 2),           # and narrower
    (1, 192, 160, 2080, 1),           # one token, the slots summed by the down product
    (1, 192, 2080, 160, 3),
    (60, 352, 320, 704, 1),
    (12, 544, 1696, 2720, 1),
])
def test_shared_experts_of_another_width(T, n_embd, n_ff, n_ff_sh, S, path):
    E, k = 5, 1 if T == 60 else 2
    st = [_experts(E, n_ff, n_embd, 1), _experts(E, n_ff, n_embd, 2), _experts(E, n_embd, n_ff, 3)]
    sh = [_experts(S, n_ff_sh, n_embd, 4), _experts(S, n_ff_sh, n_embd, 5), _experts(S, n_embd, n_ff_sh, 6)]
    dx, x = _act(T, n_embd, T)
    rng = np.random.default_rng(T + n_ff)
    ids = rng.integers(-1, E, size=(T, k)).astype(np.int32)
    rw = rng.uniform(0, 1, size=(T, k)).astype(np.float32)
    up = lambda ws: [moe.Weights(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()) for c, s, _ in ws]
    got = moe.moe_ffn_fused(*up(st), dx, dev_i32(ids), dev_f32(rw), shared=up(sh), act_quant=2, path=path)
    _check(got, *ref64.ffn(x, *(v for _, _, v in st), ids, rw, [v for _, _, v in sh]))


@pytest.mark.parametrize("path", [moe.PATH_GEMV, moe.PATH_GEMM])
def test_scale_bytes_that_start_anywhere(path):
    E, k, T, K, N = 4, 2, 20, 672, 70
    codes, scales, w = _experts(E, N, K, 5)
    dx, x = _act(T, K, 6)
    ids = np.random.default_rng(7).integers(0, E, size=(T, k)).astype(np.int32)
    ref = ref64.mul_mat_id(ref64.decode(*ref64.quantize(x)), w, ids)
    for by in (1, 2, 3, 7):
        wt = moe.Weights(torch.from_numpy(codes).cuda(), _off(torch.from_numpy(scales).cuda(), by))
        _check(moe.moe_mul_mat_id(wt, dx, dev_i32(ids), act_quant=2, path=path), *ref)
