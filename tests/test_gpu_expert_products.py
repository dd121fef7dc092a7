"""mul_mat_id with bf16, f16 and int8 experts, its gradients, and the row quantizer against their float64
forms on a GPU."""
import pytest
import torch

import indirect_expert_matmul_amd as moe
import ref_products as ref

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def _ids(T, E, k, g, segments=None, invalid=0.0, repeat=False):
    """ids [T][k]; segments: rows of each expert in turn instead of a draw (k = 1)."""
    if segments is not None:
        e = torch.repeat_interleave(torch.arange(len(segments)), torch.tensor(segments))
        return e[torch.randperm(len(e), generator=g)].to(torch.int32)[:, None].contiguous()
    if repeat:
        ids = torch.randint(0, E, (T, k), generator=g)
    else:
        ids = torch.rand((T, E), generator=g).topk(k, dim=1).indices
    ids = ids.to(torch.int32)
    if invalid:
        ids[torch.rand((T, k), generator=g) < invalid] = -1
        ids[torch.rand((T, k), generator=g) < invalid / 2] = E
    return ids.contiguous()


def _data(E, N, K, ids, dtype, per_slot, seed):
    g = torch.Generator().manual_seed(seed)
    T, k = ids.shape
    w = (torch.randn((E, N, K), generator=g) * 0.05).to(dtype)
    x = torch.randn((T * (k if per_slot else 1), K), generator=g).to(dtype)
    rw = torch.softmax(torch.randn((T, k), generator=g), 1)
    return w, x, rw


# tokens, experts, picks, N, K, rows per token, weighted, invalid ids
SHAPES = [
    (1, 4, 2, 64, 64, False, False, 0.0),
    (1, 8, 1, 1, 8, False, True, 0.0),
    (3, 5, 2, 33, 72, True, False, 0.3),
    (17, 3, 3, 130, 136, False, True, 0.2),
    (40, 2, 2, 257, 200, True, True, 0.0),
    (9, 16, 16, 95, 1048, False, False, 0.0),
    (300, 2, 1, 300, 264, False, False, 0.1),
    (513, 3, 2, 129, 328, True, True, 0.05),
    (700, 1, 1, 512, 64, False, False, 0.0),
    (120, 60, 2, 257, 328, True, True, 0.1),
    (150, 70, 2, 130, 72, False, False, 0.1),
    (500, 3, 2, 2100, 200, False, True, 0.05),
    (31, 4, 3, 100, 2120, True, False, 0.1),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,E,k,N,K,per_slot,weighted,invalid", SHAPES)
def test_product(T, E, k, N, K, per_slot, weighted, invalid, dtype):
    ids = _ids(T, E, k, torch.Generator().manual_seed(T + N), invalid=invalid)
    w, x, rw = _data(E, N, K, ids, dtype, per_slot, 1000 + K)
    out = moe.moe_mul_mat_id(moe.Weights(w.cuda()), x.cuda(), ids.cuda(), route_w=rw.cuda() if weighted else None,
                             src1_rows_per_token=k if per_slot else 1)
    y, tol = ref.product(w.double(), x.double(), ids, E, per_slot)
    if weighted:
        y, tol = ref.weighted(y, tol, rw, T, k)
    else:
        y, tol = y.view(T, k, N), tol.view(T, k, N)
    ref.within(out, y, tol, "product")


# tokens, experts, picks, N, K, rows per token, weighted, invalid ids, ids repeat
DECODE = [
    (1, 4, 2, 1, 16, False, False, 0.0, False),
    (1, 32, 4, 131, 2880, False, False, 0.0, False),
    (1, 32, 4, 131, 2880, True, True, 0.0, False),
    (8, 64, 6, 67, 1408, True, True, 0.1, False),
    (8, 64, 6, 67, 1408, False, False, 0.3, False),
    (16, 1, 4, 18, 528, False, True, 0.0, True),
    (64, 3, 1, 18, 4112, False, False, 0.1, True),
    (32, 2, 2, 5, 7184, True, True, 0.2, True),
    (5, 1024, 12, 33, 512, False, True, 0.0, False),
    (3, 7, 5, 21, 16384, False, True, 0.0, True),
]


@pytest.mark.parametrize("dtype", [BF, HF, torch.int8])
@pytest.mark.parametrize("T,E,k,N,K,per_slot,weighted,invalid,repeat", DECODE)
def test_decode(T, E, k, N, K, per_slot, weighted, invalid, repeat, dtype):
    """The GEMV path and the grouped GEMM on batches of few slots."""
    g = torch.Generator().manual_seed(T + N)
    ids = _ids(T, E, k, g, invalid=invalid, repeat=repeat)
    w, x, rw = _data(E, N, K, ids, BF if dtype == torch.int8 else dtype, per_slot, 3000 + K)
    if dtype == torch.int8:
        q, d = ref.quantize_rows(w.view(E * N, K))
        q, d = q.view(E, N, K), d.view(E, N)
        W = moe.Weights(q.to(torch.int8).cuda(), d.cuda())
        y, tol = ref.int8_product(q, d, *ref.quantize_rows(x), ids, E, per_slot)
    else:
        W = moe.Weights(w.cuda())
        y, tol = ref.product(w.double(), x.double(), ids, E, per_slot)
    if weighted:
        y, tol = ref.weighted(y, tol, rw, T, k)
    else:
        y, tol = y.view(T, k, N), tol.view(T, k, N)
    for path in (moe.PATH_GEMV, moe.PATH_GEMM):
        out = torch.full(tuple(y.shape), float("nan"), device="cuda")
        moe.moe_mul_mat_id(W, x.cuda(), ids.cuda(), route_w=rw.cuda() if weighted else None,
                           src1_rows_per_token=k if per_slot else 1, path=path, out=out)
        ref.within(out, y, tol, "path %d" % path)


SEGMENTS = [0, 1, 31, 32, 33, 63, 64, 65, 0, 127, 128, 129, 255, 256, 257, 300, 511, 513, 2]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("N,K", [(72, 136), (2100, 136), (2050, 8), (2304, 72)])
def test_product_segments(N, K, dtype):
    """Segment lengths at the tiles' edges, each expert on its own, on the narrow tiles and (wide rows of output) the
    wide ones, with one stage or a part of one too."""
    ids = _ids(0, 0, 1, torch.Generator().manual_seed(3), segments=SEGMENTS)
    E = len(SEGMENTS)
    w, x, _ = _data(E, N, K, ids, dtype, False, 5)
    out = moe.moe_mul_mat_id(moe.Weights(w.cuda()), x.cuda(), ids.cuda())
    y, tol = ref.product(w.double(), x.double(), ids, E, False)
    ref.within(out[:, 0], y, tol, "segments")


@pytest.mark.parametrize("src", [BF, HF, F32])
@pytest.mark.parametrize("T,E,k,N,K,per_slot,weighted,invalid",
                         [(s[0], s[1], s[2], s[3], (s[4] + 15) // 16 * 16) + s[5:] for s in SHAPES])
def test_int8(T, E, k, N, K, per_slot, weighted, invalid, src):
    g = torch.Generator().manual_seed(T + N + K)
    ids = _ids(T, E, k, g, invalid=invalid)
    x = (torch.randn((T * (k if per_slot else 1), K), generator=g) * 3).to(src)
    x[0] = 0
    q = torch.randint(-127, 128, (E, N, K), generator=g, dtype=torch.int8)
    d = torch.rand((E, N), generator=g) * 1e-2
    rw = torch.softmax(torch.randn((T, k), generator=g), 1)
    out = moe.moe_mul_mat_id(moe.Weights(q.cuda(), d.cuda()), x.cuda(), ids.cuda(),
                             route_w=rw.cuda() if weighted else None, src1_rows_per_token=k if per_slot else 1)
    xq, xd = ref.quantize_rows(x)
    y, tol = ref.int8_product(q, d, xq, xd, ids, E, per_slot)
    if weighted:
        y, tol = ref.weighted(y, tol, rw, T, k)
    else:
        y, tol = y.view(T, k, N), tol.view(T, k, N)
    ref.within(out, y, tol, "int8")


@pytest.mark.parametrize("N", [72, 2100])
def test_int8_segments_and_extremes(N):
    """Segment lengths at the tiles' edges; codes of -128 and 127 over the widest rows' partial stage."""
    ids = _ids(0, 0, 1, torch.Generator().manual_seed(4), segments=SEGMENTS)
    E, K = len(SEGMENTS), 272
    g = torch.Generator().manual_seed(6)
    x = torch.randn((len(ids), K), generator=g)
    q = torch.randint(-128, 128, (E, N, K), generator=g, dtype=torch.int8)
    q[3], q[4] = -128, 127
    x[:100] = 1.0
    d = torch.rand((E, N), generator=g)
    out = moe.moe_mul_mat_id(moe.Weights(q.cuda(), d.cuda()), x.cuda(), ids.cuda())
    xq, xd = ref.quantize_rows(x)
    y, tol = ref.int8_product(q, d, xq, xd, ids, E, False)
    ref.within(out[:, 0], y, tol, "int8 segments")


@pytest.mark.parametrize("src", [BF, HF, F32])
@pytest.mark.parametrize("T,k,N,K,per_slot,weighted", [(3000, 2, 40, 64, False, False), (2500, 2, 33, 80, True, True),
                                                       (1500, 3, 24, 4256, False, True), (300000, 1, 8, 16, False, False)])
def test_int8_of_many_slots(T, k, N, K, per_slot, weighted, src):
    """Codes made beside the row ids of several chunks (300000: several rows a wave), or by the quantizer's own launch."""
    g = torch.Generator().manual_seed(T)
    ids, E = _ids(T, 5, k, g, invalid=0.1), 5
    x = torch.randn((T * (k if per_slot else 1), K), generator=g).to(src)
    q = torch.randint(-127, 128, (E, N, K), generator=g, dtype=torch.int8)
    d, rw = torch.rand((E, N), generator=g) * 1e-2, torch.rand((T, k), generator=g)
    out = moe.moe_mul_mat_id(moe.Weights(q.cuda(), d.cuda()), x.cuda(), ids.cuda(), route_w=rw.cuda() if weighted else None,
                             src1_rows_per_token=k if per_slot else 1)
    y, tol = ref.int8_product(q, d, *ref.quantize_rows(x), ids, E, per_slot)
    if weighted:
        y, tol = ref.weighted(y, tol, rw, T, k)
    else:
        y, tol = y.view(T, k, N), tol.view(T, k, N)
    ref.within(out, y, tol, "int8")


@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 7), (300, 8), (70, 15), (65, 64), (33, 90), (1001, 120), (9, 121), (10, 333), (129, 512),
                                    (7, 2056), (6, 5003), (4, 7001), (5, 9000), (3, 16380), (2, 40001)])
def test_quantize_rows(rows, K, dtype):
    g = torch.Generator().manual_seed(rows + K)
    x = (torch.randn((rows, K), generator=g) * torch.exp(3 * torch.randn((rows, 1), generator=g))).to(dtype)
    q, d = moe.moe_quantize_rows(x.cuda())
    rq, rd = ref.quantize_rows(x)
    assert torch.equal(d.cpu(), rd)
    assert torch.equal(q.cpu().float(), rq)


@pytest.mark.parametrize("rows,K", [((1 << 30) + 300, 1), ((1 << 28) + 130, 9), ((1 << 24) + 9, 264), ((1 << 22) + 5, 2056)])
def test_quantize_more_rows_than_a_grid(rows, K):
    """Blocks that take several rows, each kernel's: zeros but for some rows, the first, the last and those between."""
    at = torch.tensor([0, 1, 255, 256, (1 << 22) - 1, 1 << 22, rows - 260, rows - 2, rows - 1])
    some = torch.randn((len(at), K), generator=torch.Generator().manual_seed(K)).to(BF)
    x = torch.zeros((rows, K), dtype=BF, device="cuda")
    x[at.cuda()] = some.cuda()
    q, d = moe.moe_quantize_rows(x)
    rq, rd = ref.quantize_rows(some)
    assert torch.equal(q[at.cuda()].cpu(), rq.to(torch.int8)) and torch.equal(d[at.cuda()].cpu(), rd)
    assert int((d != 0).sum()) == len(at)
    assert int(q.view(-1)[:rows * K // 8 * 8].view(torch.int64).count_nonzero()) <= 2 * len(at) * (K // 8 + 1)


def test_quantize_rows_edges():
    x = torch.zeros((8, 40))
    x[1, 5], x[2, 39] = float("inf"), float("nan")
    x[3, 0], x[4, :3] = -float("inf"), torch.tensor([127.0, 63.5, -62.5])
    x[5, :2] = torch.tensor([1e-40, -5e-41])           # subnormal scale
    x[6, 0] = 1e-45                                     # scale rounds to zero
    x[7, :2] = torch.tensor([3.4e38, -3.4e38])
    q, d = moe.moe_quantize_rows(x.cuda())
    rq, rd = ref.quantize_rows(x)
    assert torch.equal(torch.isnan(d.cpu()), torch.isnan(rd)) and torch.isnan(rd[1:4]).all()
    fine = ~torch.isnan(rd)
    assert torch.equal(d.cpu()[fine], rd[fine])
    assert torch.equal(q.cpu().float(), rq)
    assert q[4, :3].tolist() == [127, 64, -62]
    y = moe.moe_mul_mat_id(moe.Weights(torch.ones((1, 16, 48), dtype=torch.int8).cuda(), torch.ones((1, 16)).cuda()),
                           torch.nn.functional.pad(x, (0, 8)).cuda(), torch.zeros((8, 1), dtype=torch.int32).cuda())
    assert torch.equal(torch.isnan(y).all(2).flatten().cpu(), torch.isnan(rd))
    assert torch.equal(torch.isnan(y).any(2).flatten().cpu(), torch.isnan(rd))


@pytest.mark.parametrize("dtype,dw", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
@pytest.mark.parametrize("T,E,k,N,K,per_slot,weighted,invalid", SHAPES)
def test_gradients(T, E, k, N, K, per_slot, weighted, invalid, dtype, dw):
    ids = _ids(T, E, k, torch.Generator().manual_seed(T + N), invalid=invalid)
    w, x, rw = _data(E, N, K, ids, dtype, per_slot, 2000 + K)
    g = torch.Generator().manual_seed(N)
    dy = torch.randn((T, N) if weighted else (T, k, N), generator=g).to(dtype)
    got = moe.moe_mul_mat_id_backward(moe.Weights(w.cuda()), x.cuda(), ids.cuda(), dy.cuda(),
                                      route_w=rw.cuda() if weighted else None,
                                      src1_rows_per_token=k if per_slot else 1, d_w_dtype=dw)
    want = ref.grads(w.double(), x.double(), ids, dy.double(), rw if weighted else None, per_slot, dtype, dw)
    for name, a, b in zip(("d_src1", "d_w", "d_route_w"), got, want):
        if b is None:
            assert a is None
        else:
            ref.within(a, b[0].view(a.shape), b[1].view(a.shape), name)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("N,K", [(72, 40), (40, 2104), (9, 2056)])
def test_gradient_segments(N, K, dtype):
    """The row gradient on narrow and wide tiles (wide rows of src1); the experts' over more positions than its map holds."""
    ids = _ids(0, 0, 1, torch.Generator().manual_seed(8), segments=SEGMENTS + [1023, 1024, 1025])
    E = len(SEGMENTS) + 3
    w, x, rw = _data(E, N, K, ids, dtype, False, 9)
    dy = torch.randn((len(ids), 1, N), generator=torch.Generator().manual_seed(10)).to(dtype)
    got = moe.moe_mul_mat_id_backward(moe.Weights(w.cuda()), x.cuda(), ids.cuda(), dy.cuda(), d_w_dtype=F32)
    want = ref.grads(w.double(), x.double(), ids, dy.double(), None, False, dtype, F32)
    ref.within(got[0], *want[0], "d_src1")
    ref.within(got[1], *want[1], "d_w")


@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_gradients_of_wide_tiles(per_slot, weighted):
    T, E, k, N, K = 900, 8, 2, 72, 5128
    ids = _ids(T, E, k, torch.Generator().manual_seed(11), invalid=0.05)
    w, x, rw = _data(E, N, K, ids, BF, per_slot, 12)
    dy = torch.randn((T, N) if weighted else (T, k, N), generator=torch.Generator().manual_seed(13)).to(BF)
    got = moe.moe_mul_mat_id_backward(moe.Weights(w.cuda()), x.cuda(), ids.cuda(), dy.cuda(),
                                      route_w=rw.cuda() if weighted else None, src1_rows_per_token=k if per_slot else 1)
    want = ref.grads(w.double(), x.double(), ids, dy.double(), rw if weighted else None, per_slot, BF, BF)
    for name, a, b in zip(("d_src1", "d_w", "d_route_w"), got, want):
        if b is not None:
            ref.within(a, b[0].view(a.shape), b[1].view(a.shape), name)


@pytest.mark.parametrize("dtype,dw", [(BF, BF), (HF, F32)])
@pytest.mark.parametrize("segments", [[3001], [2500, 0, 1, 33, 4000, 64, 1025, 900]])
def test_gradient_of_long_segments(segments, dtype, dw):
    """Few experts of many positions: their sums in parts, some experts with fewer parts than others, or none."""
    ids = _ids(0, 0, 1, torch.Generator().manual_seed(14), segments=segments)
    E, N, K = len(segments), 75, 72
    w, x, rw = _data(E, N, K, ids, dtype, False, 15)
    dy = torch.randn((len(ids), N), generator=torch.Generator().manual_seed(16)).to(dtype)
    for weighted in (False, True):
        d = dy if weighted else dy[:, None].contiguous()
        got = moe.moe_mul_mat_id_backward(moe.Weights(w.cuda()), x.cuda(), ids.cuda(), d.cuda(),
                                          route_w=rw.cuda() if weighted else None, want=("w",), d_w_dtype=dw)[1]
        ref.within(got, *ref.grads(w.double(), x.double(), ids, d.double(), rw if weighted else None, False, dtype, dw)[1],
                   "d_w")


def test_gradients_of_many_rows():
    """More of d_dst than the thread blocks beside the row ids take at once: rounded and scaled rows of all of them."""
    T, E, N, K = 140000, 3, 1024, 16
    g = torch.Generator(device="cuda").manual_seed(21)
    ids = torch.randint(0, E, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    w = torch.randn((E, N, K), generator=g, device="cuda").to(BF)
    x = torch.randn((T, K), generator=g, device="cuda").to(BF)
    rw = torch.rand((T, 1), generator=g, device="cuda")
    dy = torch.randn((T, N), generator=g, device="cuda")
    d_x, d_w, _ = moe.moe_mul_mat_id_backward(moe.Weights(w), x, ids, dy, route_w=rw, want=("src1", "w"), d_w_dtype=F32)
    for e in range(E):
        at = torch.nonzero(ids[:, 0] == e).flatten()
        rows = (rw[at] * dy[at]).to(BF).double()          # as the library rounds them
        xe = x[at].double()
        ref.within(d_w[e], (rows.t() @ xe).cpu(), ((rows.abs().t() @ xe.abs()) * (len(at) + 1) * ref.U32).cpu(), "d_w")
        rows, we, f = dy[at].to(BF).double(), w[e].double(), rw[at].double()
        v, m = f * (rows @ we), f * (rows.abs() @ we.abs()) * (N + 1) * ref.U32
        ref.within(d_x[at], v.cpu(), ref.rounded(v, m, BF).cpu(), "d_src1")
