"""Float64 forms of mul_mat_id with 16-bit and int8 experts and of its gradients, each with a bound on
what the library's rounding may add, element by element.

A sum of n float32 products is off by at most n * 2^-24 times the sum of their magnitudes (each of the
n - 1 additions and the products' own rounding contribute at most 2^-24 of it, to first order), whatever
the order. A value stored in 16 bits is off by half a step, eps / 2 of it, or half of the smallest
subnormal."""
import torch

U32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half of the smallest subnormal."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def slots(ids, per_slot):
    """Of every slot: its expert (-1: none) and its src1 row."""
    T, k = ids.shape
    e = ids.flatten().long()
    r = torch.arange(T * k)
    return e, (r if per_slot else r // k)


def product(w, x, ids, E, per_slot):
    """(rows [n][N], bound): w [E][N][K] and x [rows][K] in float64; slots with an id outside [0, E) are 0."""
    e, r = slots(ids, per_slot)
    y = torch.zeros((len(e), w.shape[1]), dtype=torch.float64)
    m = torch.zeros_like(y)
    for i in range(E):
        at = torch.nonzero(e == i).flatten()
        y[at] = x[r[at]] @ w[i].t()
        m[at] = x[r[at]].abs() @ w[i].abs().t()
    return y, m * (w.shape[2] * U32)


def weighted(y, tol, route_w, T, k):
    """Weighted sum over the slots of float32 rows y with bound tol: k fused products, one rounding each."""
    rw = route_w.double().view(T, k, 1)
    y, tol = y.view(T, k, -1), tol.view(T, k, -1)
    return (rw * y).sum(1), (rw.abs() * tol).sum(1) + k * U32 * (rw * y).abs().sum(1)


def rounded(v, tol, dtype):
    """Bound after rounding a float32 value of v within tol to dtype."""
    return tol if dtype == torch.float32 else tol + half_step(dtype) * (v.abs() + tol) + tiny(dtype)


def grads(w, x, ids, dy, route_w, per_slot, dtype, dw_dtype):
    """((d_src1, bound), (d_w, bound), (d_route_w, bound) or None). w [E][N][K], x [rows][K] in float64; dy
    [T][k][N], weighted [T][N], as float64 values of dtype."""
    E, N, K = w.shape
    T, k = ids.shape
    e, r = slots(ids, per_slot)
    n = T * k
    rows = dy.reshape(-1, N)[torch.arange(n) // (1 if route_w is None else k)]
    valid = (e >= 0) & (e < E)
    g = torch.zeros((n, K), dtype=torch.float64)
    gt = torch.zeros_like(g)
    rw = torch.ones(n, dtype=torch.float64) if route_w is None else route_w.double().flatten()
    rw = torch.where(valid, rw, 0.0)[:, None]
    d_w = torch.zeros_like(w)
    wt = torch.zeros_like(w)
    for i in range(E):
        at = torch.nonzero(e == i).flatten()
        g[at] = rows[at] @ w[i]
        gt[at] = (rows[at].abs() @ w[i].abs()) * (N * U32)
        scaled = rows[at] * rw[at]
        d_w[i] = scaled.t() @ x[r[at]]
        # float32 sums; with weights also the scaled rows' rounding to dtype
        m = scaled.abs().t() @ x[r[at]].abs()
        once = 0.0 if route_w is None else half_step(dtype) + U32
        lost = 0.0 if route_w is None else tiny(dtype) * x[r[at]].abs().sum(0)[None, :]
        wt[i] = m * ((len(at) + 1) * U32 + once) + lost
    d_x = torch.zeros_like(x)
    xt = torch.zeros_like(x)
    d_x.index_add_(0, r, rw * g)
    xt.index_add_(0, r, rw.abs() * gt + ((1 if per_slot else k) + 1) * U32 * (rw * g).abs())
    out = [(d_x, rounded(d_x, xt, dtype)), (d_w, rounded(d_w, wt, dw_dtype)), None]
    if route_w is not None:
        xr = torch.where(valid[:, None], x[r], 0.0)
        d = (g * xr).sum(1)
        t = (gt * xr.abs()).sum(1) + K * U32 * (g * xr).abs().sum(1)
        out[2] = (d.view(T, k), t.view(T, k))
    return out


def quantize_rows(x):
    """(codes float32, scales float32) of float32 rows, decided in float32."""
    x = x.float()
    top = x.abs().amax(1)
    d = (top.double() / 127).float()
    bad = ~torch.isfinite(x).all(1)
    q = torch.round((x.double() / torch.where(d > 0, d, 1.0).double()[:, None]).float()).clamp(-127, 127)
    q = torch.where((d > 0)[:, None], q, 0.0)
    q[bad] = 0
    d = torch.where(bad, torch.nan, d)
    return q, d


def int8_product(q, d, xq, xd, ids, E, per_slot):
    """(rows, bound) of int8 experts: whole sums, then the two scales (the library rounds the sum's conversion,
    the scales' product and their product)."""
    y, _ = product(q.double(), xq.double(), ids, E, per_slot)
    e, r = slots(ids, per_slot)
    y = y * xd.double()[r][:, None] * d.double()[e.clamp(0, E - 1)]
    return y, 3.01 * U32 * y.abs()


def within(got, ref, tol, what=""):
    got = got.double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), what + ": not finite"
    off = (got - ref).abs()
    bad = off > tol
    assert not bad.any(), "%s: %d of %d values off, the worst by %.3g of what is allowed, at %s" % (
        what, int(bad.sum()), bad.numel(), float((off / tol.clamp_min(1e-300)).max()),
        torch.nonzero(bad)[0].tolist())
