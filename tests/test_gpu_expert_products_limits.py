"""16-bit and int8 expert products at the sizes where a dispatch or a kernel's grid ends."""
import pytest
import torch

import indirect_expert_matmul_amd as moe

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("dtype", [BF, torch.int8])
def test_gemv_of_rows_past_full_blocks(dtype):
    """2^25 rows in blocks of a wave for each of eight experts would be 2^32 work-items. Whole numbers: exact."""
    E, N, K = 8, (1 << 25) + 5, 8 if dtype == BF else 16
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randint(-4, 5, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
    x = torch.randint(-3, 4, (1, K), generator=g, device="cuda").to(BF)
    x[0, 0] = 127                       # int8: the row's scale is 1
    ids = torch.randperm(E, generator=g, device="cuda").to(torch.int32)[None].contiguous()
    rw = torch.exp2(torch.randint(-3, 3, (1, E), generator=g, device="cuda").float())
    want = torch.zeros(N, device="cuda")
    for s in range(E):   # column by column: the library's product of so many rows left its last ones zero
        we = w[int(ids[0, s])]
        for c in range(K):
            want += (rw[0, s] * x[0, c].float()) * we[:, c]
    W = moe.Weights(w, torch.ones((E, N), device="cuda")) if dtype == torch.int8 else moe.Weights(w.to(BF))
    assert torch.equal(moe.moe_mul_mat_id(W, x, ids, route_w=rw)[0], want)
    del W, w, want
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows,K", [((1 << 27) + 77, 40), ((1 << 26) + 41, 96), ((1 << 25) + 19, 200), ((1 << 24) + 9, 500)])
def test_quantize_more_narrow_rows_than_a_grid(rows, K):
    """Blocks that take several rows, at each number of lanes a row: zeros but for some rows."""
    at = torch.tensor([0, 1, 255, 256, (1 << 22) - 1, 1 << 22, rows - 260, rows - 2, rows - 1])
    some = torch.randn((len(at), K), generator=torch.Generator().manual_seed(K)).to(BF)
    x = torch.zeros((rows, K), dtype=BF, device="cuda")
    x[at.cuda()] = some.cuda()
    q, d = moe.moe_quantize_rows(x)
    one, scale = moe.moe_quantize_rows(some.cuda())
    assert torch.equal(q[at.cuda()], one) and torch.equal(d[at.cuda()], scale)
    assert int((d != 0).sum()) == len(at)
    del x
    assert int(q.view(-1)[:rows * K // 8 * 8].view(torch.int64).count_nonzero()) <= 2 * len(at) * (K // 8 + 1)
    del q, d
    torch.cuda.empty_cache()


def test_tensors_side_by_side():
    """Inputs and outputs that touch without sharing a byte: a call's tensors in one buffer, in two orders."""
    T, k, E, N, K = 64, 2, 4, 64, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.rand((T, E), generator=g, device="cuda").topk(k).indices.to(torch.int32)
    rw = torch.rand((T, k), generator=g, device="cuda")
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(BF)
    src, w, dy = rand(T, K), rand(E, N, K), rand(T, N)
    want = moe.moe_mul_mat_id_backward(moe.Weights(w), src, ids, dy, route_w=rw)
    shapes = dict(src=(src.shape, BF), dx=(src.shape, BF), w=(w.shape, BF), dw=(w.shape, BF), rw=(rw.shape, torch.float32),
                  dr=(rw.shape, torch.float32), dy=(dy.shape, BF))
    for order in (list(shapes), list(shapes)[::-1]):
        buf, at, t = torch.empty(1 << 20, dtype=torch.uint8, device="cuda"), 0, {}
        for n in order:
            shape, dt = shapes[n]
            size = shape.numel() * dt.itemsize
            t[n] = buf[at:at + size].view(dt).view(shape)
            at += size
        for n, v in (("src", src), ("w", w), ("rw", rw), ("dy", dy)):
            t[n].copy_(v)
        moe.moe_mul_mat_id_backward(moe.Weights(t["w"]), t["src"], ids, t["dy"], route_w=t["rw"], d_src1=t["dx"], d_w=t["dw"],
                                    d_route_w=t["dr"])
        for a, b in zip(want, (t["dx"], t["dw"], t["dr"])):
            assert torch.equal(a, b)
    with pytest.raises(moe.MoeError, match="overlap"):
        moe.moe_mul_mat_id_backward(moe.Weights(w), src, ids, dy, route_w=rw, d_route_w=rw)
    x = torch.randn((33, 40), generator=g, device="cuda")
    q, d = moe.moe_quantize_rows(x)
    buf = torch.empty(33 * 40 * 5 + 33 * 4, dtype=torch.uint8, device="cuda")
    buf[33 * 4:33 * 164].view(torch.float32).view(33, 40).copy_(x)
    p = buf.data_ptr()
    assert moe.lib.moe_quantize_rows(p + 33 * 4, moe.MOE_F32, 33, 40, p + 33 * 164, p, None) == moe.MOE_OK
    torch.cuda.synchronize()
    assert torch.equal(buf[:33 * 4].view(torch.float32), d) and torch.equal(buf[33 * 164:].view(torch.int8).view(33, 40), q)
