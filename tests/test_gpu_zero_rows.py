"""Per-slot output of moe_mul_mat_id: rows of slots whose id is out of range are zero and nothing around
the output is touched, on every path, for rows of one column to several pieces of a wave's columns."""
import numpy as np
import pytest
import torch

import indirect_expert_matmul_amd as moe

pytestmark = pytest.mark.gpu


def _experts(kind, E, N, K):
    g = torch.Generator().manual_seed(N)
    if kind == "f32":
        return moe.Weights(torch.randn((E, N, K), generator=g).cuda())
    if kind == "q8":
        return moe.Weights(torch.randint(-127, 128, (E, N, K), dtype=torch.int8, generator=g).cuda(),
                           torch.full((E, N, K // 32), 0.01, dtype=torch.float16).cuda())
    return moe.Weights(torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, generator=g).cuda(),
                       torch.full((E, N, K // 32), 120, dtype=torch.uint8).cuda())


@pytest.mark.parametrize("kind,path,aq", [("f32", 0, 0), ("q8", moe.PATH_GEMM, 0), ("q8", moe.PATH_GEMV, 0),
                                          ("q8", moe.PATH_GEMM, 1), ("mxfp4", moe.PATH_GEMM, 0),
                                          ("mxfp4", moe.PATH_GEMM, 2), ("mxfp4", moe.PATH_GEMV, 2)])
@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (3, 3, 2047), (5, 2, 2048), (1, 9, 2051), (4, 4, 10001)])
@pytest.mark.parametrize("bad", [0.6, 1.0])
def test_rows_of_invalid_slots(kind, path, aq, T, k, N, bad):
    E, K = 3, 128
    w = _experts(kind, E, N, K)
    rng = np.random.default_rng(T + N)
    ids = rng.integers(0, E, size=(T, k)).astype(np.int32)
    off = rng.random((T, k)) < bad
    off[0, 0] = True
    ids[off] = rng.choice((-1, E, E + 7, -2 ** 31, 2 ** 31 - 1), size=off.sum())
    x = torch.randn((T, K), generator=torch.Generator().manual_seed(1)).cuda()
    x = x if kind == "f32" else x.to(torch.bfloat16)
    buf = torch.full((64 + T * k * N + 64,), 7.0, device="cuda")
    out = buf[64:64 + T * k * N].view(T, k, N)
    out.fill_(float("nan"))
    moe.moe_mul_mat_id(w, x, torch.from_numpy(ids).cuda(), out=out, path=path, act_quant=aq)
    torch.cuda.synchronize()
    o = out.cpu().numpy()
    assert np.all(o[off] == 0) and np.all(np.isfinite(o))
    assert N < 100 or np.all((o[~off] != 0).any(axis=1))
    assert (buf[:64] == 7).all() and (buf[64 + T * k * N:] == 7).all()


@pytest.mark.parametrize("kind,path,aq", [("f32", 0, 0), ("q8", moe.PATH_GEMM, 0), ("mxfp4", moe.PATH_GEMM, 2)])
def test_more_slots_than_one_group_a_thread_block(kind, path, aq):
    """Past 2^21 slots each thread block takes several groups of them."""
    E, K, N, T, k = 5, 32, 3, 300007, 9
    assert T * k > 2 ** 21
    w = _experts(kind, E, N, K)
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.randint(-2, E + 2, (T, k), dtype=torch.int32, device="cuda", generator=g)
    x = torch.randn((T, K), device="cuda", generator=g) + 0.5
    x = x if kind == "f32" else x.to(torch.bfloat16)
    out = torch.full((T, k, N), float("nan"), device="cuda")
    moe.moe_mul_mat_id(w, x, ids, out=out, path=path, act_quant=aq)
    off = (ids < 0) | (ids >= E)
    assert (out[off] == 0).all() and torch.isfinite(out).all()
    assert (out[~off] != 0).any(dim=1).float().mean() > 0.99
