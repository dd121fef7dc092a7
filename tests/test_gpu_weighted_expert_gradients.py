"""The experts' gradient of weighted calls, d_w[e] = sum of w_i * dy_i (outer) x_i, at the precision of its sums: the
factors are not rounded to the experts' type on the way.

Bounds. The rows v = w_i * dy_i (float32, off by U32 of v) go to the products in parts whose sum is off by at most
PART[dtype] of v (two parts, the first cut off and the second rounded: 2^-7 * 2^-8 for bfloat16's 8 bits, 2^-10 * 2^-11
for float16's 11; three parts, for a float32 result, hold all 24 bits). float16 rows are scaled by a power of two that
puts the call's largest |v| of a slot with an expert within [2^14, 2^15]: the last part is off by at most one smallest
subnormal, 2^-24, which is at most 2^-38 of that largest one. The sums add (n + 1) * U32."""
import pytest
import torch

import indirect_expert_matmul_amd as moe
import ref_products as ref

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
PART = {BF: 2.0 ** -15, HF: 2.0 ** -21}


def _call(T=77, E=5, k=2, N=75, K=72, dtype=BF, per_slot=False, invalid=0.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand((T, E), generator=g).topk(k, dim=1).indices.to(torch.int32)
    if invalid:
        ids[torch.rand((T, k), generator=g) < invalid] = -1
        ids[torch.rand((T, k), generator=g) < invalid / 2] = E
    w = (torch.randn((E, N, K), generator=g) * 0.05).to(dtype)
    x = torch.randn((T * (k if per_slot else 1), K), generator=g).to(dtype)
    rw = torch.softmax(torch.randn((T, k), generator=g), 1)
    dy = torch.randn((T, N), generator=g).to(dtype)
    return w, x, ids, dy, rw, per_slot


def _d_w(w, x, ids, dy, rw, per_slot, dw, **kw):
    return moe.moe_mul_mat_id_backward(moe.Weights(w.cuda()), x.cuda(), ids.cuda(), dy.cuda(), route_w=rw.cuda(),
                                       src1_rows_per_token=ids.shape[1] if per_slot else 1, want=("w",), d_w_dtype=dw, **kw)[1]


def _bounds(w, x, ids, dy, rw, per_slot, dw):
    """d_w in float64 and what it may be off by."""
    E, N, K = w.shape
    e, r = ref.slots(ids, per_slot)
    k = ids.shape[1]
    v = dy.double()[torch.arange(len(e)) // k] * rw.double().flatten()[:, None]
    valid = (e >= 0) & (e < E)
    top = v[valid].abs().max() if valid.any() else 0.0
    parts = 2 if dw != F32 else 3
    d, tol = torch.zeros((E, N, K), dtype=torch.float64), torch.zeros((E, N, K), dtype=torch.float64)
    for i in range(E):
        at = torch.nonzero(e == i).flatten()
        xe = x.double()[r[at]]
        d[i] = v[at].t() @ xe
        tol[i] = v[at].abs().t() @ xe.abs() * ((parts * len(at) + 2) * ref.U32 + (PART[w.dtype] if dw != F32 else 0.0))
        if w.dtype == HF:
            tol[i] += 2.0 ** -38 * top * xe.abs().sum(0)[None, :]
    return d, ref.rounded(d, tol, dw)


@pytest.mark.parametrize("dtype,dw", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
@pytest.mark.parametrize("T,E,k,N,K,per_slot,invalid", [(1, 1, 1, 1, 8, False, 0.0), (17, 3, 3, 130, 136, True, 0.2),
                                                        (77, 5, 2, 75, 72, False, 0.1), (513, 3, 2, 129, 328, True, 0.05),
                                                        (700, 1, 1, 300, 264, False, 0.0), (120, 60, 2, 257, 328, False, 0.0),
                                                        (3000, 2, 2, 64, 40, False, 0.1)])
@pytest.mark.parametrize("f32", [False, True])
def test_rows_keep_their_bits(T, E, k, N, K, per_slot, invalid, dtype, dw, f32):
    w, x, ids, dy, rw, per_slot = _call(T, E, k, N, K, dtype, per_slot, invalid, T + N)
    if f32:   # a float32 d_dst is multiplied as it is
        dy = torch.randn((T, N), generator=torch.Generator().manual_seed(N))
    got = _d_w(w, x, ids, dy, rw, per_slot, dw)
    ref.within(got, *_bounds(w, x, ids, dy, rw, per_slot, dw), "d_w")


@pytest.mark.parametrize("f32", [False, True])
def test_float32_d_dst_with_weights(f32):
    """Of a float32 d_dst, weighted d_w takes the factors' products with the unrounded rows; d_src1 and d_route_w the rows
    rounded to the experts' type."""
    w, x, ids, _, rw, per_slot = _call(seed=3)
    dy = torch.randn((len(ids), w.shape[1]), generator=torch.Generator().manual_seed(4))
    dd = dy if f32 else dy.to(BF)
    got = moe.moe_mul_mat_id_backward(moe.Weights(w.cuda()), x.cuda(), ids.cuda(), dd.cuda(), route_w=rw.cuda())
    same = moe.moe_mul_mat_id_backward(moe.Weights(w.cuda()), x.cuda(), ids.cuda(), dy.to(BF).cuda(), route_w=rw.cuda())
    assert torch.equal(got[0], same[0]) and torch.equal(got[2], same[2])
    ref.within(got[1], *_bounds(w, x, ids, dd, rw, per_slot, BF), "d_w")


@pytest.mark.parametrize("dtype,dw", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
def test_infinities_stay_infinities(dtype, dw):
    """An infinity in src1 or d_dst gives infinities of the right sign where nothing is zero, and only in its column or row."""
    w, x, ids, dy, rw, per_slot = _call(dtype=dtype, seed=11)
    dy = torch.where(dy.abs() < 2.0 ** -6, 2.0 ** -6, dy.float()).to(dtype)   # no zeros, some with few bits
    dy[3] = torch.tensor([1.0, -1.0, 0.5]).repeat(25).to(dtype)
    rw[3] = torch.tensor([0.5, 0.25])                                        # products of one bit
    clean = _d_w(w, x, ids, dy, rw, per_slot, dw)
    xi = x.clone()
    xi[3, 5] = float("inf")
    got = _d_w(w, xi, ids, dy, rw, per_slot, dw).cpu()
    for s in range(2):
        e = int(ids[3, s])
        assert torch.equal(got[e, :, 5].float(), torch.where(dy[3].float() > 0, float("inf"), -float("inf")))
        got[e, :, 5] = clean[e, :, 5].cpu()
    assert torch.equal(got, clean.cpu())
    di = dy.clone()
    di[3, 7] = -float("inf")
    xs = torch.where(x.abs() < 2.0 ** -6, 2.0 ** -6, x.float()).to(dtype)
    clean = _d_w(w, xs, ids, dy, rw, per_slot, dw).cpu()
    got = _d_w(w, xs, ids, di, rw, per_slot, dw).cpu()
    for s in range(2):
        e = int(ids[3, s])
        assert torch.equal(got[e, 7].float(), torch.where(xs[3].float() > 0, -float("inf"), float("inf")))
        got[e, 7] = clean[e, 7]
    assert torch.equal(got, clean)
