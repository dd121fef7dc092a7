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
