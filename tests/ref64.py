"""Scored routing, its gradient, MXFP4 quantization and products of MXFP4 tensors written out
in float64 numpy, with the error bounds the GPU tests hold float32 results to. Shares no
code with the library.

Bounds count roundings: float32 is off by at most EPS = 2^-24 relative per operation.
"""
import numpy as np

EPS = 2.0 ** -24
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])


# ---------------------------------------------------------------- scored routing
def scores(logits, kind):
    """float64 scores; logits of -inf or NaN have score 0 and stay out of the softmax's sum."""
    l = np.asarray(logits, np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    s = np.zeros_like(l)
    for t in range(l.shape[0]):
        row = l[t]
        top = row.max()
        if kind == "sigmoid":
            with np.errstate(over="ignore"):
                s[t] = 1 / (1 + np.exp(-row))
        elif top == np.inf:
            s[t] = (row == np.inf) / np.sum(row == np.inf)
        elif top > -np.inf:
            z = np.exp(row - top)
            s[t] = z / z.sum()
    return s


def pick_weights(l, s, kind, renorm, scale):
    """Weights of one token's picks with logits l and scores s, renormalised without 0 / 0."""
    if not renorm:
        return scale * s
    if len(l) == 0:
        return s
    top = l.max()
    if kind == "sigmoid":
        log_s = -np.logaddexp(0.0, -l)
        r = np.exp(log_s - log_s.max())
    elif top == np.inf:
        r = (l == np.inf).astype(np.float64)
    else:
        r = np.exp(l - top)
    return scale * r / r.sum()


def route(logits, k, bias=None, score="softmax", n_group=1, topk_group=1, group_top=2, renorm=True, scale=1.0):
    """(ids int32 [T][k], weights float64 [T][k], scores float64 [T][E])."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    s = scores(l, score)
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
    ok_bias = ~np.isnan(b) & (b != -np.inf)
    for t in range(T):
        ok = ~np.isnan(l[t]) & (l[t] != -np.inf) & ok_bias
        choice = l[t] if bias is None else s[t] + b
        order = s[t] if bias is None and group_top == 2 else choice    # what group scores sum
        best = []
        for g in range(n_group):
            m = [e for e in range(g * E // n_group, (g + 1) * E // n_group) if ok[e]]
            if m:
                best.append((-sum(sorted((order[e] for e in m), reverse=True)[:group_top]), g))
        kept = {g for _, g in sorted(best)[:topk_group]} if topk_group < n_group else set(range(n_group))
        live = [e for e in range(E) if ok[e] and e * n_group // E in kept]
        live.sort(key=lambda e: (-choice[e], e))
        p = live[:k]
        ids[t, :len(p)] = p
        w[t, :len(p)] = pick_weights(l[t, p], s[t, p], score, renorm, scale)
    return ids, w, s


def route_backward(logits, ids, d_w, d_s=None, score="softmax", renorm=True, scale=1.0):
    """(d_logits float64 [T][E], bound [T][E] on a float32 evaluation's error)."""
    l = np.asarray(logits, np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    T, E = l.shape
    s = scores(l, score)
    out, bound = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        js = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E and l[t, ids[t, j]] > -np.inf]
        es = ids[t, js]
        w = pick_weights(l[t, es], s[t, es], score, renorm, 1.0)
        g = np.asarray(d_w[t, js], np.float64)
        mean, mean_abs = (w @ g, w @ np.abs(g)) if renorm else (0.0, 0.0)
        q, mag = np.zeros(E), np.zeros(E)                       # s_e dL/ds_e
        np.add.at(q, es, scale * w * (g - mean))
        np.add.at(mag, es, abs(scale) * w * (np.abs(g) + mean_abs))
        if d_s is not None:
            r = d_s if d_s.ndim == 1 else d_s[t]
            live = l[t] > -np.inf
            q[live] += s[t, live] * r[live]
            mag[live] += s[t, live] * np.abs(r[live])
        if score == "softmax":
            out[t] = q - s[t] * q.sum()
            mag = mag + s[t] * mag.sum()
        else:
            with np.errstate(over="ignore"):
                rest = 1 / (1 + np.exp(l[t]))
            out[t], mag = q * rest, mag * rest
        out[t][l[t] == -np.inf] = 0
        bound[t] = rounding(l[t], E + ids.shape[1]) * mag
    return out, bound


def rounding(l, terms):
    """Relative error of a float32 score, weight or product of them: an exponential of a difference of
    logits carries the difference's rounding (|difference| EPS, at most twice the largest logit), twice
    (numerator and sum); a sum of `terms` values in any order at most terms EPS; 32 more for the
    exponentials, quotients and products themselves."""
    f = l[np.isfinite(l)]
    span = 2 * np.abs(f).max() if f.size else 0.0
    return (2 * span + terms + 32) * EPS


# ---------------------------------------------------------------- MXFP4
def quantize(x):
    """(codes uint8 [rows][K] one per element, scale bytes uint8 [rows][K/32]) of float values."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[0], -1, 32)
    bad = ~np.isfinite(b).all(axis=2)
    v = np.where(bad[:, :, None], 0.0, b)
    top = np.abs(v).max(axis=2)
    _, e = np.frexp(top)                                        # top = m 2^e, m in [1/2, 1)
    byte = np.where(top > 0, np.maximum(e - 1 - 2 + 127, 0), 0)
    code = nearest(np.ldexp(v, (127 - byte)[:, :, None]))
    code[bad] = 0
    byte[bad] = 255
    return code.reshape(x.shape), byte.astype(np.uint8)


def nearest(v):
    """E2M1 code of the value nearest to v, ties to the even code, saturated."""
    a = np.abs(v)[..., None]
    grid = E2M1[:8]
    d = np.abs(a - grid)
    tie = d == d.min(axis=-1, keepdims=True)
    even = tie & (np.arange(8) % 2 == 0)
    m = np.where(even.any(axis=-1), even.argmax(axis=-1), tie.argmax(axis=-1))
    return (m | (np.signbit(v).astype(np.int64) << 3)).astype(np.uint8)


def pack(codes):
    return (codes[..., ::2] | codes[..., 1::2] << 4).astype(np.uint8)


def unpack(packed):
    return np.stack((packed & 15, packed >> 4), axis=-1).reshape(packed.shape[:-1] + (-1,))


def decode(codes, byte):
    """float64 values of one code per element and one scale byte per 32."""
    s = np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))
    v = E2M1[codes].reshape(codes.shape[:-1] + (-1, 32)) * s[..., None]
    return v.reshape(codes.shape)


def product_bound(K):
    """Error of a float32 sum of K products relative to the sum of their magnitudes: one rounding per
    128 columns (the matrix instruction's own sum and the accumulator), doubled for its inner order."""
    return 2 * (K / 128 + 2) * EPS


def mul_mat_id(x, w, ids, route_w=None, B=1):
    """(out, bound): x [T*B][K] and w [E][N][K] float64 values."""
    T, k = ids.shape
    E, N, K = w.shape
    y, a = np.zeros((T, k, N)), np.zeros((T, k, N))
    for t in range(T):
        for s in range(k):
            e = ids[t, s]
            if 0 <= e < E:
                r = x[t * B + s % B]
                y[t, s] = w[e] @ r
                a[t, s] = np.abs(w[e]) @ np.abs(r)
    if route_w is None:
        return y, product_bound(K) * a
    ok = ((ids >= 0) & (ids < E))[:, :, None]
    rw = np.asarray(route_w, np.float64)[:, :, None]
    return (np.where(ok, rw * y, 0).sum(axis=1),
            np.where(ok, (product_bound(K) + (k + 1) * EPS) * np.abs(rw) * a, 0).sum(axis=1))


def ffn(x, gate, up, down, ids, route_w, shared=None):
    """(out, bound) of the fused FFN on MXFP4 activations: x bf16/float values [T][n_embd], the expert
    stacks as float64 values. h is quantized from values known up to their float32 error, so the bound
    adds, for each element of h, how far its code's value can move within that error."""
    xq = decode(*quantize(x))
    T, k = ids.shape
    out, bound = np.zeros((T, down.shape[1])), np.zeros((T, down.shape[1]))

    def expert(t, g, u, d, weight):
        r, ra = xq[t], np.abs(xq[t])
        gv, uv = g @ r, u @ r
        eg, eu = (product_bound(len(r)) * (np.abs(m) @ ra) for m in (g, u))
        silu = gv / (1 + np.exp(-gv))
        h = silu * uv
        dh = 1.1 * eg * np.abs(uv) + np.abs(silu) * eu + 1.1 * eg * eu + 16 * (1 + np.abs(gv)) * EPS * np.abs(h)
        hq = decode(*quantize(h[None]))[0]
        b, db = np.abs(h).reshape(-1, 32), dh.reshape(-1, 32)
        lo, hi = hq.copy(), hq.copy()
        for top in ((b - db).max(axis=1), (b + db).max(axis=1)):  # the block's scale, at either end
            _, e = np.frexp(np.maximum(top, 0))
            byte = np.where(top > 0, np.maximum(e - 1 - 2 + 127, 0), 0)
            for v in (h - dh, h + dh):
                z = np.ldexp(v.reshape(-1, 32), (127 - byte)[:, None])
                q = decode(nearest(z).reshape(1, -1), byte[None].astype(np.uint8))[0]
                lo, hi = np.minimum(lo, q), np.maximum(hi, q)
        y, a = d @ hq, np.abs(d) @ np.maximum(np.abs(lo), np.abs(hi))
        out[t] += weight * y
        bound[t] += abs(weight) * ((product_bound(len(h)) + (k + 4) * EPS) * a + np.abs(d) @ (hi - lo))

    for t in range(T):
        for s in range(k):
            if 0 <= ids[t, s] < gate.shape[0]:
                e = ids[t, s]
                expert(t, gate[e], up[e], down[e], float(route_w[t, s]))
        for j in range(shared[0].shape[0] if shared else 0):
            expert(t, shared[0][j], shared[1][j], shared[2][j], 1.0)
    return out, bound
