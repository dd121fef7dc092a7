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
