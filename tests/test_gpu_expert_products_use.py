"""16-bit and int8 expert products, their gradients and the row quantizer as programs use them: a training step and a
decode step of a whole layer, on several streams, in captured graphs, with used workspaces of exactly the size asked
for, on tensors whose offsets pass 32 bits, and with infinities and NaN in some rows."""
import pytest
import torch

import indirect_expert_matmul_amd as moe
import ref_products as ref

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _same(a, b):
    assert a.shape == b.shape and a.dtype == b.dtype
    kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    differ = (a.contiguous().view(kind) != b.contiguous().view(kind)).sum().item()
    assert differ == 0, "%d of %d values differ" % (differ, a.numel())


def _ids(T, E, k, invalid=0.0):
    ids = torch.rand((T, E), device="cuda").topk(k).indices.to(torch.int32)
    if invalid:
        ids[torch.rand((T, k), device="cuda") < invalid] = -1
    return ids


def _weights(E, N, K, dtype):
    if dtype == torch.int8:
        return moe.Weights(torch.randint(-127, 128, (E, N, K), dtype=torch.int8, device="cuda"),
                           torch.rand((E, N), device="cuda") * 1e-3)
    return moe.Weights((torch.randn((E, N, K), device="cuda") * 0.05).to(dtype))


# ---------------------------------------------------------------- a layer's steps
class Training:
    """Scored routing, gate and up products, silu(gate) * up, weighted down product, and all gradients."""

    def __init__(self, T, seed, E=8, k=3, n_embd=136, n_ff=72, dtype=BF):
        torch.manual_seed(seed)
        self.k, self.dtype = k, dtype
        self.gate, self.up = _weights(E, n_ff, n_embd, dtype), _weights(E, n_ff, n_embd, dtype)
        self.down = _weights(E, n_embd, n_ff, dtype)
        self.x = torch.randn((T, n_embd), device="cuda").to(dtype)
        self.logits = torch.randn((T, E), device="cuda")
        if T > 4:
            self.logits[T // 2] = -float("inf")   # padding: no expert
        self.d_out = torch.randn((T, n_embd), device="cuda").to(dtype)

    def run(self, **kw):
        k, x = self.k, self.x
        ids, rw = moe.moe_router_scored(self.logits, k, renorm=True, scale=1.5, **kw)
        g, u = moe.moe_mul_mat_id(self.gate, x, ids, **kw), moe.moe_mul_mat_id(self.up, x, ids, **kw)
        s = torch.sigmoid(g)
        h = (g * s * u).to(self.dtype)
        out = moe.moe_mul_mat_id(self.down, h, ids, route_w=rw, src1_rows_per_token=k, **kw)
        d_h, d_down, d_rw = moe.moe_mul_mat_id_backward(self.down, h, ids, self.d_out, route_w=rw, src1_rows_per_token=k,
                                                        d_w_dtype=F32, **kw)
        f = d_h.float()
        d_g, d_u = (f * u * s * (1 + g * (1 - s))).to(self.dtype), (f * g * s).to(self.dtype)
        dx_g, d_gate, _ = moe.moe_mul_mat_id_backward(self.gate, x, ids, d_g, **kw)
        dx_u, d_up, _ = moe.moe_mul_mat_id_backward(self.up, x, ids, d_u, **kw)
        d_logits = moe.moe_router_scored_backward(self.logits, ids, d_rw, renorm=True, scale=1.5, **kw)
        return dict(ids=ids, rw=rw, g=g, u=u, h=h, out=out, d_h=d_h, d_down=d_down, d_rw=d_rw, d_g=d_g, d_u=d_u,
                    dx_g=dx_g, d_gate=d_gate, dx_u=dx_u, d_up=d_up, d_logits=d_logits)


@pytest.mark.parametrize("T,dtype", [(1, BF), (20, HF), (300, BF)])
def test_training_step(T, dtype):
    """Every product and gradient of the step against its float64 form on the tensors that it got; the whole
    step's gradients against autograd in float64."""
    a = Training(T, 3, dtype=dtype)
    r = {n: t.cpu() for n, t in a.run().items()}
    W = {n: getattr(a, n).data.cpu().double() for n in ("gate", "up", "down")}
    E, k, ids, x = 8, a.k, r["ids"], a.x.cpu().double()
    for name, got in (("gate", r["g"]), ("up", r["u"])):
        y, tol = ref.product(W[name], x, ids, E, False)
        ref.within(got.view(T * k, -1), y, tol, name)
    h = r["h"].double().view(T * k, -1)
    y, tol = ref.product(W["down"], h, ids, E, True)
    ref.within(r["out"], *ref.weighted(y, tol, r["rw"], T, k), "down")
    for name, xx, dy, rw, dw, got in (("down", h, a.d_out.cpu(), r["rw"], F32, ("d_h", "d_down", "d_rw")),
                                      ("gate", x, r["d_g"], None, dtype, ("dx_g", "d_gate")),
                                      ("up", x, r["d_u"], None, dtype, ("dx_u", "d_up"))):
        want = ref.grads(W[name], xx, ids, dy.double(), rw, name == "down", dtype, dw)
        for n, w in zip(got, want):
            ref.within(r[n].view(w[0].shape), w[0], w[1], n)
    # the whole step: gradients of sum(out * d_out), experts without a token and padding tokens included
    P = {n: W[n].clone().requires_grad_(True) for n in W}
    xa, la = x.clone().requires_grad_(True), a.logits.cpu().double().clone().requires_grad_(True)
    p = torch.softmax(torch.where(torch.isinf(la).all(1, keepdim=True), torch.zeros_like(la), la), 1)
    loss = 0.0
    for t in range(T):
        if ids[t, 0] < 0:
            continue
        e = ids[t].long()
        w = p[t, e] / p[t, e].sum() * 1.5
        hid = torch.nn.functional.silu(P["gate"][e] @ xa[t]) * (P["up"][e] @ xa[t])
        loss = loss + (w[:, None] * (P["down"][e] @ hid[:, :, None])[:, :, 0] * a.d_out[t].cpu().double()).sum()
    loss.backward()
    # Six tensors on the way are rounded to 16 bits, each by at most 2^-8 of itself (bf16): the results' error stays
    # near sqrt(6) * 2^-8 = 0.0096 of them while roundings are independent, and under 6 * 2^-8 = 0.0235 if not.
    for got, want in ((r["dx_g"].double() + r["dx_u"].double(), xa.grad), (r["d_gate"].double(), P["gate"].grad),
                      (r["d_up"].double(), P["up"].grad), (r["d_down"].double(), P["down"].grad),
                      (r["d_logits"].double(), torch.nan_to_num(la.grad))):
        assert (got - want).norm() <= 0.0235 * want.norm() + 1e-12


@pytest.mark.parametrize("given", [False, True])
def test_training_steps_on_streams(given):
    layers = [Training(300, 1), Training(40, 2, dtype=HF), Training(1100, 3)]
    refs = [a.run() for a in layers]
    torch.cuda.synchronize()
    if given:   # the calls' stream argument, with another one current: the products alone (torch's own work would not follow)
        st = [torch.cuda.Stream() for _ in layers]
        for _ in range(5):
            outs = []
            for a, s, r in zip(layers, st, refs):
                outs.append(moe.moe_mul_mat_id_backward(a.down, r["h"], r["ids"], a.d_out, route_w=r["rw"],
                                                        src1_rows_per_token=a.k, d_w_dtype=F32, stream=s))
                outs[-1] += (moe.moe_mul_mat_id(a.gate, a.x, r["ids"], stream=s),)
            torch.cuda.synchronize()
            for o, r in zip(outs, refs):
                for n, t in zip(("d_h", "d_down", "d_rw", "g"), o):
                    _same(t, r[n])
        return
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(5):
        outs = []
        for a, s in zip(layers, streams):
            with torch.cuda.stream(s):
                outs.append(a.run())
        torch.cuda.synchronize()
        for o, r in zip(outs, refs):
            for n in r:
                _same(o[n], r[n])


def test_training_steps_in_two_graphs():
    """Two captured steps replayed in turn, with eager work between, on new inputs each time."""
    layers = [Training(30, 1), Training(400, 2, dtype=HF)]
    graphs, outs = [], []
    for a in layers:
        a.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(a.run())
        graphs.append(g)
    eager = Training(100, 3)
    for i in range(5):
        for a in layers:
            a.x.normal_()
            a.logits.normal_()
            a.d_out.normal_()
        order = (0, 1) if i % 2 else (1, 0)
        for j in order:
            graphs[j].replay()
            eager.run()
        torch.cuda.synchronize()
        for a, o in zip(layers, outs):
            want = a.run()
            torch.cuda.synchronize()
            for n in want:
                _same(o[n], want[n])


@pytest.mark.parametrize("T,dtype", [(1, torch.int8), (6, torch.int8), (1, BF), (40, torch.int8)])
def test_decode_steps_in_a_graph(T, dtype):
    """A decode step through int8 (made by the row quantizer) or bf16 experts, captured and replayed on new tokens."""
    torch.manual_seed(T)
    E, k, n_embd, n_ff = 16, 4, 528, 272

    def experts(N, K):
        w = torch.randn((E, N, K), device="cuda") * 0.05
        return moe.Weights(*moe.moe_quantize_rows(w)) if dtype == torch.int8 else moe.Weights(w.to(dtype))
    up, down = experts(n_ff, n_embd), experts(n_embd, n_ff)
    x = torch.randn((T, n_embd), device="cuda").to(BF)
    logits = torch.randn((T, E), device="cuda")

    def step():
        ids, rw = moe.moe_router_topk(logits, k)
        h = torch.nn.functional.silu(moe.moe_mul_mat_id(up, x, ids)).to(BF)
        return ids, rw, h, moe.moe_mul_mat_id(down, h, ids, route_w=rw, src1_rows_per_token=k)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(5):
        x.normal_()
        logits.normal_()
        g.replay()
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            _same(a, b)
    ids, rw, h, out = (t.cpu() for t in got)
    if dtype == torch.int8:
        y, tol = ref.int8_product(down.data.cpu(), down.scales.cpu(), *ref.quantize_rows(h.view(T * k, n_ff)), ids, E, True)
    else:
        y, tol = ref.product(down.data.cpu().double(), h.double().view(T * k, n_ff), ids, E, True)
    ref.within(out, *ref.weighted(y, tol, rw, T, k), "down")


# ---------------------------------------------------------------- workspaces and bounds
def _guarded(nbytes):
    """A workspace of exactly nbytes, used, and the bytes behind it."""
    t = torch.full((nbytes + 4096,), 255, dtype=torch.uint8, device="cuda")
    t[nbytes:] = 171
    return t[:nbytes], t[nbytes:]


@pytest.mark.parametrize("T,E,k,N,K,per_slot", [(3, 4, 2, 37, 48, False), (9, 5, 3, 40, 64, True), (400, 6, 2, 333, 272, False),
                                                (700, 3, 2, 260, 528, True), (600, 8, 2, 5000, 5136, True), (600, 8, 2, 5001, 5136, False)])
def test_workspace_of_the_size_asked_for(T, E, k, N, K, per_slot):
    """Used workspaces of exactly the reported size, outputs in guarded buffers; ten identical runs."""
    torch.manual_seed(T)
    B = k if per_slot else 1
    ids, rw = _ids(T, E, k, 0.1), torch.rand((T, k), device="cuda")
    x = torch.randn((T * B, K), device="cuda").to(BF)
    for w in (_weights(E, N, K, BF), _weights(E, N, K, torch.int8)):
        for weighted in (False, True):
            for path in (moe.PATH_GEMM, moe.PATH_GEMV) if T * k <= 64 else (moe.PATH_GEMM,):
                need = moe.moe_mul_mat_id_workspace_size(w, moe.MOE_BF16, B, T, k, path=path)
                first = None
                for _ in range(3):
                    ws, behind = _guarded(need)
                    out = torch.full((T + 2,) + ((N,) if weighted else (k, N)), 7.0, device="cuda")
                    moe.moe_mul_mat_id(w, x, ids, route_w=rw if weighted else None, src1_rows_per_token=B, path=path,
                                       out=out[1:T + 1], workspace=ws)
                    assert (behind == 171).all() and (out[0] == 7).all() and (out[T + 1] == 7).all()
                    first = out if first is None else first
                    _same(out, first)
                assert torch.isfinite(first).all()
    w = _weights(E, N, K, BF)
    for weighted in (False, True):
        dy = torch.randn((T, N) if weighted else (T, k, N), device="cuda").to(BF)
        for want in (("src1",), ("w",), ("src1", "w")) + ((("route_w",), ("src1", "w", "route_w")) if weighted else ()):
            for dd in (dy, dy.float()):
                need = moe.moe_mul_mat_id_backward_workspace_size(w, moe.MOE_F32 if dd is not dy else moe.MOE_BF16, B, T, k,
                                                                  weighted, want)
                first = None
                for _ in range(3):
                    ws, behind = _guarded(need)
                    dx = torch.full((T * B + 2, K), 7.0, device="cuda", dtype=BF)
                    dw = torch.full((E + 2, N, K), 7.0, device="cuda", dtype=F32)
                    got = moe.moe_mul_mat_id_backward(
                        w, x, ids, dd, route_w=rw if weighted else None, src1_rows_per_token=B, want=want,
                        d_src1=dx[1:-1] if "src1" in want else None, d_w=dw[1:-1] if "w" in want else None, workspace=ws)
                    assert (behind == 171).all()
                    for t in (dx, dw):
                        assert (t[0] == 7).all() and (t[-1] == 7).all()
                    assert [t is not None for t in got] == [n in want for n in ("src1", "w", "route_w")]
                    got = [t.clone() for t in got if t is not None]
                    first = got if first is None else first
                    for a, b in zip(got, first):
                        assert torch.isfinite(a).all()
                        _same(a, b)


def test_gradient_of_float32_and_misplaced_d_dst():
    """float32 d_dst is d_dst rounded once; a d_dst off 16-byte alignment, or with odd rows, is copied."""
    torch.manual_seed(5)
    for N in (72, 75):
        T, E, k, K = 50, 4, 2, 64
        ids, w, x = _ids(T, E, k), _weights(E, N, K, BF), torch.randn((T, K), device="cuda").to(BF)
        dy = torch.randn((T, k, N), device="cuda")
        a = moe.moe_mul_mat_id_backward(w, x, ids, dy.to(BF))
        b = moe.moe_mul_mat_id_backward(w, x, ids, dy)
        off = torch.empty(T * k * N + 1, dtype=BF, device="cuda")
        off[1:] = dy.to(BF).flatten()
        c = moe.moe_mul_mat_id_backward(w, x, ids, off[1:].view(T, k, N))
        for u, v, z in zip(a[:2], b[:2], c[:2]):
            _same(u, v)
            _same(u, z)


def test_no_tokens():
    w = _weights(3, 40, 64, BF)
    x, ids = torch.empty((0, 64), dtype=BF, device="cuda"), torch.empty((0, 2), dtype=torch.int32, device="cuda")
    assert moe.moe_mul_mat_id(w, x, ids).shape == (0, 2, 40)
    dw = torch.full((3, 40, 64), 7.0, device="cuda", dtype=BF)
    d = moe.moe_mul_mat_id_backward(w, x, ids, torch.empty((0, 2, 40), dtype=BF, device="cuda"), d_w=dw)
    assert d[0].shape == (0, 64) and (dw == 0).all()
    q, s = moe.moe_quantize_rows(x)
    assert q.shape == (0, 64) and s.shape == (0,)


def test_no_expert_at_all():
    """Every id invalid: rows of zeros, gradients of zeros."""
    T, k = 70, 2
    x, ids = torch.randn((T, 64), device="cuda").to(BF), torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    rw = torch.rand((T, k), device="cuda")
    for w in (_weights(3, 40, 64, BF), _weights(3, 40, 64, torch.int8)):
        for t in (1, T):
            assert (moe.moe_mul_mat_id(w, x[:t], ids[:t]) == 0).all()
            assert (moe.moe_mul_mat_id(w, x[:t], ids[:t], route_w=rw[:t].contiguous()) == 0).all()
    d = moe.moe_mul_mat_id_backward(_weights(3, 40, 64, BF), x, ids, torch.randn((T, 40), device="cuda").to(BF), route_w=rw)
    assert all((t == 0).all() for t in d)


# ---------------------------------------------------------------- infinities and NaN
@pytest.mark.parametrize("T", [5, 200])
def test_bad_rows_stay_their_own(T):
    """NaN in one token's activations, in one expert and in one row of d_dst reach only what they are part of; an
    infinity gives infinities, not NaN, next to the zeros that fill up a segment's last stage."""
    torch.manual_seed(T)
    E, k, N, K = 6, 2, 71, 72
    ids, w = _ids(T, E, k), _weights(E, N, K, BF)
    x, dy = torch.randn((T, K), device="cuda").to(BF), torch.randn((T, k, N), device="cuda").to(BF)
    paths = (moe.PATH_GEMM, moe.PATH_GEMV) if T * k <= 64 else (moe.PATH_GEMM,)
    clean = [moe.moe_mul_mat_id(w, x, ids, path=p) for p in paths]
    dclean = moe.moe_mul_mat_id_backward(w, x, ids, dy)
    bad_t, bad_e = T // 2, int(ids[0, 0])
    xb = x.clone()
    xb[bad_t, K - 1] = float("nan")
    for p, c in zip(paths, clean):
        y = moe.moe_mul_mat_id(w, xb, ids, path=p)
        assert torch.isnan(y[bad_t]).all()
        keep = torch.arange(T, device="cuda") != bad_t
        _same(y[keep], c[keep])
    wb = moe.Weights(w.data.clone())
    wb.data[bad_e, N - 1, 0] = float("nan")
    for p, c in zip(paths, clean):
        y = moe.moe_mul_mat_id(wb, x, ids, path=p)
        hit = (ids == bad_e)[:, :, None] & (torch.arange(N, device="cuda") == N - 1)
        assert torch.equal(torch.isnan(y), hit)
        assert torch.equal(y[~hit], c[~hit])
    # gradients
    dyb = dy.clone()
    dyb[bad_t, 1, 3] = float("nan")
    dx, dw, _ = moe.moe_mul_mat_id_backward(w, x, ids, dyb)
    keep = torch.arange(T, device="cuda") != bad_t
    assert torch.isnan(dx[bad_t]).all()
    _same(dx[keep], dclean[0][keep])
    e = int(ids[bad_t, 1])
    hit = (torch.arange(E, device="cuda") == e)[:, None, None] & (torch.arange(N, device="cuda") == 3)[:, None]
    assert torch.equal(torch.isnan(dw), hit.expand_as(dw))
    xi = x.clone()
    xi[bad_t, 5] = float("inf")
    dw = moe.moe_mul_mat_id_backward(w, xi, ids, dy, want=("w",))[1]
    assert (dy[bad_t] != 0).all()
    for s in range(k):
        got = dw[int(ids[bad_t, s]), :, 5].float()
        assert torch.equal(got, torch.where(dy[bad_t, s].float() > 0, float("inf"), -float("inf")))
    assert torch.isfinite(dw[:, :, :5].float()).all() and torch.isfinite(dw[:, :, 6:].float()).all()


def test_subnormal_halves():
    """float16 subnormals count on both paths and in the gradients."""
    E, N, K = 2, 40, 64
    w = moe.Weights(torch.full((E, N, K), 2.0 ** -24, dtype=HF, device="cuda"))
    x = torch.full((6, K), 2.0 ** -20, dtype=HF, device="cuda")
    ids = torch.tensor([[0], [1], [0], [1], [0], [1]], dtype=torch.int32, device="cuda")
    for p in (moe.PATH_GEMM, moe.PATH_GEMV):
        assert (moe.moe_mul_mat_id(w, x, ids, path=p) == 64 * 2.0 ** -44).all()
    dy = torch.full((6, 1, N), 2.0 ** -10, dtype=HF, device="cuda")
    dx, dw, _ = moe.moe_mul_mat_id_backward(w, x, ids, dy, d_w_dtype=F32)
    assert (dw == 3 * 2.0 ** -30).all()
    assert (dx == torch.tensor(40 * 2.0 ** -34, dtype=HF, device="cuda")).all()


# ---------------------------------------------------------------- offsets past 32 bits
@pytest.mark.parametrize("dtype", [BF, torch.int8])
@pytest.mark.parametrize("T,path", [(7, moe.PATH_GEMV), (7, moe.PATH_GEMM), (300, moe.PATH_GEMM)])
def test_experts_past_32_bits(T, path, dtype):
    """Over 2^32 weights, of which the last two experts are used."""
    E, N, K = 37, 8192, 16384
    w = moe.Weights(torch.empty((E, N, K), dtype=dtype, device="cuda"),
                    torch.rand((E, N), device="cuda") if dtype == torch.int8 else None)
    assert w.data.numel() > 2 ** 32
    w.data[E - 2:] = torch.randint(-9, 10, (2, N, K), device="cuda", dtype=torch.int8).to(dtype)
    x = torch.randn((T, K), device="cuda").to(BF)
    ids = _ids(T, 2, 2)
    tail = moe.Weights(w.data[E - 2:], None if w.scales is None else w.scales[E - 2:])
    a = moe.moe_mul_mat_id(tail, x, ids, path=path)
    b = moe.moe_mul_mat_id(w, x, ids + (E - 2), path=path)
    if dtype == BF and path == moe.PATH_GEMM:
        # the numbers of experts may take tiles that add in different orders: each float32 sum of K products is off by
        # at most K 2^-24 of the sum of their magnitudes, so the two differ by at most twice that
        for e in range(2):
            t, s = torch.nonzero(ids == e, as_tuple=True)
            most = 2 * K * 2.0 ** -24 * (x[t].double().abs() @ tail.data[e].double().abs().t())
            assert ((a[t, s].double() - b[t, s].double()).abs() <= most).all()
    else:
        _same(a, b)
    assert a.abs().max() > 0
    if dtype == BF and path == moe.PATH_GEMM:
        dy = torch.randn((T, 2, N), device="cuda").to(BF)
        a = moe.moe_mul_mat_id_backward(tail, x, ids, dy)
        b = moe.moe_mul_mat_id_backward(w, x, ids + (E - 2), dy)
        _same(a[0], b[0])
        _same(a[1], b[1][E - 2:])
        assert (b[1][:E - 2] == 0).all() and a[1].abs().max() > 0


@pytest.mark.parametrize("dtype", [BF, torch.int8])
def test_rows_past_32_bits(dtype):
    """Activations, outputs and gradient rows of over 2^32 bytes and 2^31 elements."""
    T, E, N, K, n = 270001, 3, 8200, 8208, 400
    w = _weights(E, N, K, dtype)
    x = torch.empty((T, K), dtype=BF, device="cuda")
    x.normal_()
    ids = _ids(T, E, 1)
    assert T * K > 2 ** 31 and T * N > 2 ** 31
    out = moe.moe_mul_mat_id(w, x, ids)
    for at in (0, T // 2, T - n):
        _same(out[at:at + n], moe.moe_mul_mat_id(w, x[at:at + n], ids[at:at + n], path=moe.PATH_GEMM))
    if dtype == torch.int8:
        return
    dy = out.to(BF)
    del out
    rw = torch.rand((T, 1), device="cuda")
    for weighted in (False, True):
        d = dy.view(T, N) if weighted else dy
        got = moe.moe_mul_mat_id_backward(w, x, ids, d, route_w=rw if weighted else None,
                                          want=("src1", "route_w") if weighted else ("src1",))
        for at in (0, T // 2, T - n):
            s = slice(at, at + n)
            part = moe.moe_mul_mat_id_backward(w, x[s], ids[s], d[s].contiguous(), route_w=rw[s].contiguous() if weighted else None,
                                               want=("src1", "route_w") if weighted else ("src1",))
            _same(got[0][s], part[0])
            if weighted:
                # d_route_w's sum of K products is split by the tiles of the call, which its size decides: two results
                # are apart by at most twice K roundings of 2^-24 of the sum of their magnitudes (the rows of g from
                # d_src1, whose rounding is 2^-8 of them)
                g = part[0].double().abs() / rw[s].double()
                tol = 2 * K * ref.U32 * (1 + 2.0 ** -7) * (g * x[s].double().abs()).sum(1, keepdim=True)
                assert ((got[2][s].double() - part[2].double()).abs() <= tol).all()
    # the experts' gradients from rows past 32 bits: only the last tokens have an expert
    few = torch.full_like(ids, -1)
    few[T - n:] = ids[T - n:]
    for weighted in (False, True):
        d = dy.view(T, N) if weighted else dy
        big = moe.moe_mul_mat_id_backward(w, x, few, d, route_w=rw if weighted else None, want=("w",))[1]
        s = slice(T - n, T)
        _same(big, moe.moe_mul_mat_id_backward(w, x[s], ids[s], d[s].contiguous(), route_w=rw[s].contiguous() if weighted else None,
                                               want=("w",))[1])


@pytest.mark.parametrize("dtype,K", [(BF, 4104), (F32, 2052), (BF, 16392)])
def test_quantize_past_32_bits(dtype, K):
    base = 4099
    rep = 2 ** 32 // (base * K) + 1
    x = (torch.randn((base, K), device="cuda") * torch.rand((base, 1), device="cuda") * 9).to(dtype)
    q, d = moe.moe_quantize_rows(x)
    Q, D = moe.moe_quantize_rows(x.repeat(rep, 1))
    assert Q.numel() > 2 ** 32
    assert (Q.view(rep, base, K) == q).all() and (D.view(rep, base) == d).all()


def test_many_short_rows():
    """More rows than one grid takes a wave each, and rows shorter than a load."""
    for K in (3, 16):
        x = torch.randn((4099, K), device="cuda")
        rep = 2 ** 24 // 4099 + 9
        q, d = moe.moe_quantize_rows(x)
        Q, D = moe.moe_quantize_rows(x.repeat(rep, 1))
        assert (Q.view(rep, 4099, K) == q).all() and (D.view(rep, 4099) == d).all()
