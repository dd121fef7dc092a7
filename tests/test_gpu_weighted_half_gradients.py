"""float16 experts: products of routing weights and gradients that leave float16's range, in the experts' gradient."""
import pytest
import torch

import indirect_expert_matmul_amd as moe
import ref_products as ref
from test_gpu_weighted_expert_gradients import BF, F32, HF, _bounds, _call, _d_w

pytestmark = pytest.mark.gpu


RANGE = [(2.0 ** -12, 2.0 ** -14), (1e-3, 1e-4), (2.5, 4e4), (2.0 ** -40, 2.0 ** -20), (2.0 ** -100, 2.0 ** -3)]
PAST = [(3e4, 6e4), (2.0 ** 60, 1.0)]   # no float16 result holds these


@pytest.mark.parametrize("factor,size,dw", [r + (d,) for r in RANGE for d in (HF, F32)] + [r + (F32,) for r in PAST])
def test_products_past_the_range(factor, size, dw):
    """All slots' factors near one size and all gradients near another: against the sum of magnitudes, without the rows'
    rounding to float16's subnormals. (x is small, so that sums fit a float16 result, or large, so that they are not lost
    in it.)"""
    w, x, ids, dy, rw, per_slot = _call(dtype=HF, seed=int(size > 1))
    rw = factor * (1 + torch.rand(rw.shape, generator=torch.Generator().manual_seed(1)))
    dy = (size * (0.5 + 0.5 * dy.float().clamp(-1, 1))).to(HF)
    if dw == HF:
        x = (x.float() * (2.0 ** -7 if factor > 1 else 2.0 ** 9)).to(HF)
    got = _d_w(w, x, ids, dy, rw, per_slot, dw)
    d, tol = _bounds(w, x, ids, dy, rw, per_slot, dw)
    fits = d.abs() + tol < torch.finfo(dw).max
    assert fits.all()
    ref.within(got, d, tol, "d_w")


def test_float32_rows_past_the_range():
    """A float32 d_dst of numbers that float16 has not, small factors beside large ones."""
    w, x, ids, _, rw, per_slot = _call(dtype=HF, seed=5)
    g = torch.Generator().manual_seed(6)
    for size in (1e-12, 1e9):
        dy = torch.randn((len(ids), w.shape[1]), generator=g) * size
        rw = rw * torch.exp2(-10 * torch.rand(rw.shape, generator=g))
        got = _d_w(w, x, ids, dy, rw, per_slot, F32)
        ref.within(got, *_bounds(w, x, ids, dy, rw, per_slot, F32), "d_w")


def test_slots_without_an_expert_do_not_scale():
    """Rows of padding, which may hold anything, have no part in the scale."""
    w, x, ids, dy, rw, per_slot = _call(dtype=HF, seed=7)
    clean = _d_w(w, x, ids, dy, rw, per_slot, F32)
    for bad_w, bad_dy in ((1e30, 1.0), (1.0, 6e4), (float("inf"), 1.0), (float("nan"), float("nan"))):
        i2 = torch.cat((ids, torch.full((3, 2), -1, dtype=torch.int32)))
        i2[-1] = w.shape[0]
        r2 = torch.cat((rw, torch.full((3, 2), bad_w)))
        d2 = torch.cat((dy, torch.full((3, dy.shape[1]), bad_dy, dtype=HF)))
        x2 = torch.cat((x, torch.zeros((3, x.shape[1]), dtype=HF)))
        assert torch.equal(_d_w(w, x2, i2, d2, r2, per_slot, F32), clean)


def test_zeros_and_no_experts():
    w, x, ids, dy, rw, per_slot = _call(dtype=HF, seed=8)
    assert (_d_w(w, x, ids, torch.zeros_like(dy), rw, per_slot, F32) == 0).all()
    assert (_d_w(w, x, torch.full_like(ids, -1), dy, rw, per_slot, HF) == 0).all()
    none = [t[:0] for t in (x, ids, dy, rw)]
    assert (_d_w(w, none[0], none[1], none[2], none[3], per_slot, F32) == 0).all()
    ids[ids == 2] = -1   # an expert without slots
    got = _d_w(w, x, ids, dy, rw, per_slot, F32)
    assert (got[2] == 0).all() and got.abs().max() > 0


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,E,k,N,K,per_slot", [(9, 5, 3, 40, 64, True), (700, 3, 2, 260, 528, False), (2600, 2, 2, 75, 72, True)])
def test_used_workspace_of_the_size_asked_for(T, E, k, N, K, per_slot, dtype):
    """Workspaces of exactly the reported size full of NaN, with either type of d_w; the same bits each time."""
    w, x, ids, dy, rw, per_slot = _call(T, E, k, N, K, dtype, per_slot, 0.1, 13)
    W, B = moe.Weights(w.cuda()), k if per_slot else 1
    x, ids, dy, rw = x.cuda(), ids.cuda(), dy.cuda(), rw.cuda()
    for want in (("w",), ("src1", "w", "route_w")):
        for dw in (dtype, F32):
            for dd in (dy, dy.float()):
                need = moe.moe_mul_mat_id_backward_workspace_size(W, moe._elem_type(dd), B, T, k, True, want)
                first = None
                for _ in range(3):
                    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
                    got = moe.moe_mul_mat_id_backward(W, x, ids, dd, route_w=rw, src1_rows_per_token=B, want=want, d_w_dtype=dw,
                                                      workspace=ws[:need])
                    assert (ws[need:] == 255).all()
                    first = got if first is None else first
                    for a, b in zip(got, first):
                        assert a is b or torch.equal(a, b)
                    assert all(torch.isfinite(t).all() for t in got if t is not None)


def test_two_captured_gradients_in_turn():
    """Gradients of both types captured, replayed on new inputs of another size of numbers each time (the scale is the
    replay's own), with eager calls between."""
    calls, graphs, outs = [], [], []
    for i, (dtype, dw) in enumerate(((HF, HF), (BF, BF), (HF, F32))):
        w, x, ids, dy, rw, _ = _call(300, 5, 2, 75, 72, dtype, False, 0.1, 20 + i)
        a = dict(W=moe.Weights(w.cuda()), x=x.cuda(), ids=ids.cuda(), dy=dy.cuda(), rw=rw.cuda(), dw=dw)

        def run(a=a):
            return moe.moe_mul_mat_id_backward(a["W"], a["x"], a["ids"], a["dy"], route_w=a["rw"], d_w_dtype=a["dw"])
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run())
        calls.append((a, run))
        graphs.append(g)
    for r in range(5):
        for a, _ in calls:
            a["dy"].normal_().mul_(2.0 ** (3 * r - 8))
            a["rw"].uniform_().mul_(2.0 ** (-4 * r))
            a["x"].normal_()
        for j in ((0, 1, 2), (2, 0, 1))[r % 2]:
            graphs[j].replay()
            calls[(j + 1) % 3][1]()
        torch.cuda.synchronize()
        for (a, run), o in zip(calls, outs):
            for u, v in zip(run(), o):
                assert torch.equal(u, v) and torch.isfinite(u).all() and u.abs().max() > 0


def test_top_of_many_tokens():
    """More tokens than the blocks that look for the largest product take one of; the largest is in the last row."""
    w, x, ids, dy, rw, per_slot = _call(9001, 3, 1, 16, 8, HF, False, 0.0, 31)
    dy[-1, -1] = 6e4
    rw = rw * 1e-3
    rw[-1] = 2.0
    ref.within(_d_w(w, x, ids, dy, rw, per_slot, F32), *_bounds(w, x, ids, dy, rw, per_slot, F32), "d_w")


@pytest.mark.parametrize("dw", [HF, F32])
def test_small_products_beside_a_large_one(dw):
    """Columns of d_dst whose numbers, of a few bits, are 2^-26 to 2^-36 of another column's: relative to their own size
    off by the roundings of float32 sums and of the result (a whole number of units of 2^-24 is a sum of two such)."""
    T, E, k, N, K = 60, 2, 1, 24, 16
    g = torch.Generator().manual_seed(40)
    ids = torch.randint(0, E, (T, k), generator=g).to(torch.int32)
    w = torch.zeros((E, N, K), dtype=HF)
    x = torch.randint(1, 4, (T, K), generator=g).to(HF)
    dy = torch.randint(1, 8, (T, N), generator=g).double() * torch.exp2(-torch.arange(N).double() - 12)
    dy[:, 0] = 6.0 * 2 ** 12
    dy, rw = dy.to(HF), torch.exp2(-torch.randint(0, 2, (T, k), generator=g).float())
    got = _d_w(w, x, ids, dy, rw, False, dw).double().cpu()
    v = dy.double() * rw.double()
    top = v.max()
    for e in range(E):
        at = torch.nonzero(ids[:, 0] == e).flatten()
        want = v[at].t() @ x[at].double()
        tol = want * 3 * len(at) * ref.U32 + (ref.half_step(HF) * want + ref.tiny(HF) if dw == HF else 0)
        big = (v[at] >= 2 * top * 2.0 ** -38).all(0)   # at least three units
        assert big.sum() >= 10
        past = want - tol >= torch.finfo(dw).max   # 24576 of every slot: a float16 result's sum is infinite
        assert torch.equal(torch.isinf(got[e]), past) and past.any() == (dw == HF)
        assert (past | ((got[e] - want).abs() <= tol))[big].all()
