"""GPU parity of MXFP4 quantization and of the products of MXFP4 activations with MXFP4 experts
(act_quant = 2) against the float64 forms of ref64: codes, scale bytes and values equal; products
within the float32 summation bound of ref64.product_bound; the FFN within that bound plus how far
the codes of h can move inside h's own float32 error."""
import numpy as np
import pytest
import torch

import indirect_expert_matmul_amd as moe
import ref64
import synth
from moe_testutil import dev_f32, dev_i32

pytestmark = pytest.mark.gpu


def _values(rows, K, seed):
    """float32 rows of very different size with blocks at the format's edges."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, K)) * np.exp(rng.uniform(-3, 3, size=(rows, 1)))
    b = x.reshape(rows, -1, 32)
    n = b.shape[1]
    edges = [
        np.zeros(32), -np.zeros(32),
        np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.99, -0.25, -5.0, 4.0, -0.1, 0.3, 2.0], 2),
        np.concatenate(([2.0 ** 127 * 1.75], rng.standard_normal(31))),           # the largest exponent
        np.concatenate(([2.0 ** -126], rng.uniform(-1, 1, 31) * 2.0 ** -126)),    # smallest normal maximum
        rng.uniform(-1, 1, 32) * 2.0 ** -130,                                     # subnormal maximum
        rng.uniform(-4, 4, 32) * 2.0 ** -124,
    ]
    for i, v in enumerate(edges):
        if i < rows * n:
            b[i // n, i % n] = v
    return x.astype(np.float32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (7, 2880), (65, 1056), (300, 2048), (2, 16384)])
def test_quantize_equal(rows, K, dtype):
    x = torch.from_numpy(_values(rows, K, rows + K)).to(dtype)
    codes, scales, values = moe.moe_quantize_mxfp4(x.cuda(), return_values=True)
    c2, s2 = moe.moe_quantize_mxfp4(x.cuda())
    torch.cuda.synchronize()
    rc, rb = ref64.quantize(x.double().numpy())
    assert np.array_equal(codes.cpu().numpy(), ref64.pack(rc))
    assert np.array_equal(scales.cpu().numpy(), rb)
    assert torch.equal(c2, codes) and torch.equal(s2, scales)
    want = torch.from_numpy(ref64.decode(rc, rb))
    assert values.dtype == dtype
    bits = torch.int16 if dtype == torch.bfloat16 else torch.int32
    assert torch.equal(values.cpu().view(bits), want.to(dtype).view(bits))   # signs of zero included


def test_quantize_non_finite_blocks_in_place_and_empty():
    x = torch.from_numpy(_values(4, 128, 3))
    x[0, 5], x[1, 40], x[2, 127] = float("inf"), float("nan"), -float("inf")
    codes, scales, values = moe.moe_quantize_mxfp4(x.cuda(), return_values=True)
    rc, rb = ref64.quantize(x.double().numpy())
    assert np.array_equal(codes.cpu().numpy(), ref64.pack(rc)) and np.array_equal(scales.cpu().numpy(), rb)
    assert (rb == 255).sum() == 3
    want = ref64.decode(rc, rb).astype(np.float32)
    assert np.array_equal(values.cpu().numpy(), want, equal_nan=True)
    buf = x.cuda()
    moe.lib.moe_quantize_mxfp4(buf.data_ptr(), moe.MOE_F32, 4, 128, codes.data_ptr(), scales.data_ptr(),
                               buf.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert np.array_equal(buf.cpu().numpy(), want, equal_nan=True)
    c, s = moe.moe_quantize_mxfp4(torch.zeros((0, 64), device="cuda"))
    assert c.shape == (0, 32) and s.shape == (0, 2)
    w = torch.from_numpy(_values(6, 64, 1)).view(2, 3, 64).cuda()
    c, s = moe.moe_quantize_mxfp4(w)
    assert c.shape == (2, 3, 32) and s.shape == (2, 3, 2)
    assert moe.Weights(c, s).type == moe.MOE_MXFP4


def _experts(E, N, K, seed, lo=118, hi=122):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, size=(E, N, K // 2), dtype=np.uint8)
    scales = rng.integers(lo, hi, size=(E, N, K // 32), dtype=np.uint8)
    return codes, scales, ref64.decode(ref64.unpack(codes), scales)


def _upload(codes, scales):
    return moe.Weights(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())


def _act(rows, K, seed):
    """bf16 activations and their float64 values."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, K)) * np.exp(rng.uniform(-2, 2, size=(rows, 1)))
    t = torch.from_numpy(x).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def _check(got, ref, bound):
    g = got.cpu().numpy().astype(np.float64)
    err = np.abs(g - ref)
    assert np.all(err <= bound + 1e-37), "off by %.3g over a bound of %.3g" % ((err - bound).max(), bound.max())


def _mul_mat_id(E, k, T, K, N, B, ids, path, lo=118, hi=122):
    codes, scales, w = _experts(E, N, K, K + N, lo, hi)
    dx, x = _act(T * B, K, T + K)
    xq = ref64.decode(*ref64.quantize(x))
    wt = _upload(codes, scales)
    rng = np.random.default_rng(T)
    rw = rng.standard_normal((T, k)).astype(np.float32)
    got = moe.moe_mul_mat_id(wt, dx, dev_i32(ids), src1_rows_per_token=B, act_quant=2, path=path)
    gotw = moe.moe_mul_mat_id(wt, dx, dev_i32(ids), route_w=dev_f32(rw), src1_rows_per_token=B, act_quant=2,
                              path=path)
    torch.cuda.synchronize()
    _check(got, *ref64.mul_mat_id(xq, w, ids, None, B))
    _check(gotw, *ref64.mul_mat_id(xq, w, ids, rw, B))
    g = got.cpu().numpy()
    assert np.all(g[(ids < 0) | (ids >= E)] == 0.0)
    again = moe.moe_mul_mat_id(wt, dx, dev_i32(ids), src1_rows_per_token=B, act_quant=2, path=path)
    torch.cuda.synchronize()
    assert torch.equal(again.view(torch.int32), got.view(torch.int32))


@pytest.mark.parametrize("E,k,T,K,N,B_is_k,routing", [
    (6, 3, 9, 96, 40, False, "bad"),        # K ends inside a stage; ragged N; invalid ids
    (16, 2, 50, 256, 300, True, "uniform"), # one src1 row per slot
    (4, 4, 300, 544, 513, False, "bad"),    # several M tiles per expert, odd N
    (8, 2, 400, 1024, 256, False, "zipf"),  # skewed segments: empty, tiny and oversized
    (3, 2, 1, 64, 64, False, "uniform"),    # a single token
    (1, 1, 129, 32, 1, False, "uniform"),   # one block of K, one column
    (4, 6, 70, 160, 130, True, "repeat"),   # the same expert in several slots
    (5, 2, 600, 2880, 96, False, "uniform"),
    (2, 1, 33, 7168, 64, False, "uniform"),
    (8, 2, 30, 128, 64, False, "none"),     # every id invalid
    (8, 4, 2600, 160, 72, False, "bad"),    # row ids over several thread blocks
    (700, 3, 40, 128, 33, True, "bad"),     # more experts than the row-id pass's mask words
    (900, 5, 1900, 96, 24, False, "bad"),
])
def test_mul_mat_id_grouped(E, k, T, K, N, B_is_k, routing):
    rng = np.random.default_rng(T * 31 + E)
    if routing == "zipf":
        ids = synth.draw_ids_zipf(3, T, E, k, 1.1)
    elif routing == "repeat":
        ids = rng.integers(0, E, size=(T, k)).astype(np.int32)
    elif routing == "none":
        ids = np.full((T, k), -1, np.int32)
    else:
        ids = synth.draw_ids_uniform(3, T, E, k)
    if routing == "bad":
        ids[0, 0], ids[T - 1, k - 1] = -1, E + 2
    _mul_mat_id(E, k, T, K, N, k if B_is_k else 1, ids, moe.PATH_GEMM)


@pytest.mark.parametrize("E,k,T,K,N,B_is_k,routing", [
    (3, 2, 1, 128, 64, False, "uniform"),    # one token, the shortest rows
    (32, 4, 1, 2880, 2880, False, "uniform"),# one token, GPT-OSS-shaped
    (32, 4, 8, 2880, 200, True, "uniform"),  # several slots an expert, K ends inside a superstep
    (4, 2, 32, 544, 33, False, "uniform"),   # 64 slots, up to 32 of one expert, odd N
    (1, 1, 64, 160, 17, False, "uniform"),   # 64 slots of one expert
    (1, 2, 31, 192, 5, True, "repeat"),      # the same expert in both slots
    (2, 1, 3, 16416, 16, False, "uniform"),  # several rounds of two supersteps a wave
    (16, 4, 5, 4096, 48, False, "bad"),
    (256, 8, 2, 7168, 40, False, "uniform"), # wide rows
    (1000, 7, 9, 1056, 16, False, "uniform"),
    (8, 2, 9, 128, 64, False, "none"),       # every id invalid
])
def test_mul_mat_id_gemv(E, k, T, K, N, B_is_k, routing):
    rng = np.random.default_rng(T * 31 + E)
    if routing == "repeat":
        ids = rng.integers(0, E, size=(T, k)).astype(np.int32)
    elif routing == "none":
        ids = np.full((T, k), -1, np.int32)
        ids[3] = E
    else:
        ids = synth.draw_ids_uniform(3, T, E, k)
    if routing == "bad":
        ids[0, 0], ids[T - 1, k - 1] = -1, E + 2
        ids[2] = -7
    _mul_mat_id(E, k, T, K, N, k if B_is_k else 1, ids, moe.PATH_GEMV)
    assert moe.last_stage_count() == 1      # unweighted: one launch


@pytest.mark.parametrize("path", [moe.PATH_GEMM, moe.PATH_GEMV])
def test_mul_mat_id_wide_scales_and_nan_scale(path):
    """Scales over most of the E8M0 range and a NaN scale in one expert row."""
    ids = synth.draw_ids_uniform(4, 30, 4, 2)
    _mul_mat_id(4, 2, 30, 256, 96, 1, ids, path, lo=60, hi=190)
    codes, scales, _ = _experts(4, 96, 256, 9)
    scales[2, 17, 3] = 255
    w = ref64.decode(ref64.unpack(codes), scales)
    dx, x = _act(30, 256, 2)
    dx[11, 70] = float("inf")
    got = moe.moe_mul_mat_id(_upload(codes, scales), dx, dev_i32(ids), act_quant=2, path=path).cpu().numpy()
    ref, _ = ref64.mul_mat_id(ref64.decode(*ref64.quantize(dx.double().cpu().numpy())), w, ids)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.isnan(ref[11]).all() and np.isnan(ref).mean() < 0.2


@pytest.mark.parametrize("rows", [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 160, 200])
def test_segment_lengths(rows):
    """One expert with `rows` rows next to others with a few."""
    T = rows + 5
    ids = np.full((T, 1), 2, np.int32)
    ids[rows:, 0] = [0, 1, 3, 3, 0]
    _mul_mat_id(4, 1, T, 288, 160, 1, ids, moe.PATH_GEMM)


def _ffn_case(E, k, T, n_embd, n_ff, S, ids, path=moe.PATH_AUTO):
    st = [_experts(E, n_ff, n_embd, 1), _experts(E, n_ff, n_embd, 2), _experts(E, n_embd, n_ff, 3)]
    sh = [_experts(S, n_ff // 2 * 2, n_embd, 4), _experts(S, n_ff // 2 * 2, n_embd, 5),
          _experts(S, n_embd, n_ff, 6)] if S else None
    t = torch.from_numpy(np.random.default_rng(7).standard_normal((T, n_embd))).to(torch.bfloat16)
    rw = np.random.default_rng(8).uniform(0, 1, size=ids.shape).astype(np.float32)
    dev = [_upload(c, s) for c, s, _ in st]
    dsh = [_upload(c, s) for c, s, _ in sh] if S else None
    got = moe.moe_ffn_fused(*dev, t.cuda(), dev_i32(ids), dev_f32(rw), shared=dsh, act_quant=2, path=path)
    torch.cuda.synchronize()
    ref, bound = ref64.ffn(t.double().numpy(), *(v for _, _, v in st), ids, rw, [v for _, _, v in sh] if S else None)
    _check(got, ref, bound)
    # the bound is what float32 can move, not a licence: most elements sit far inside it
    print("ffn error %.3g of max, bound %.3g" % (np.abs(got.cpu().numpy() - ref).max() / np.abs(ref).max(),
                                                 bound.max() / np.abs(ref).max()))
    return got, dev, dsh, t, rw


@pytest.mark.parametrize("E,k,T,n_embd,n_ff,S,routing", [
    (8, 2, 12, 96, 64, 0, "uniform"),       # K tails on both projections
    (8, 3, 40, 256, 160, 2, "bad"),         # shared experts, ragged N tiles, invalid ids
    (6, 2, 200, 512, 768, 1, "zipf"),       # skewed segments, several M tiles
    (4, 6, 10, 64, 32, 1, "repeat"),        # n_used > n_experts: duplicate experts
    (4, 2, 1, 352, 96, 1, "uniform"),       # one token
])
def test_ffn(E, k, T, n_embd, n_ff, S, routing):
    ids = (synth.draw_ids_zipf(23, T, E, k, 1.1) if routing == "zipf"
           else np.random.default_rng(T * 31 + E).integers(0, E, size=(T, k)).astype(np.int32))
    if routing == "bad":
        ids[0, 0], ids[5] = -1, E
    _ffn_case(E, k, T, n_embd, n_ff, S, ids, path=moe.PATH_GEMM)
    assert moe.last_stage_count() == 4      # row ids with the quantization of x, gate/up, down, reduce


@pytest.mark.parametrize("E,k,T,n_embd,n_ff,S,routing", [
    (8, 2, 12, 160, 128, 0, "uniform"),
    (8, 3, 20, 256, 160, 2, "bad"),
    (4, 6, 10, 128, 256, 1, "repeat"),
    (4, 2, 1, 352, 192, 1, "uniform"),
    (16, 4, 1, 2880, 1440, 0, "uniform"),
    (3, 1, 64, 544, 128, 1, "uniform"),     # 64 slots and 64 shared rows
    (6, 2, 3, 128, 192, 3, "none"),         # only the shared experts
])
def test_ffn_gemv(E, k, T, n_embd, n_ff, S, routing):
    ids = np.random.default_rng(T * 31 + E).integers(0, E, size=(T, k)).astype(np.int32)
    if routing == "bad":
        ids[0, 0], ids[5] = -1, E
    if routing == "none":
        ids[:] = -1
    got, *rest = _ffn_case(E, k, T, n_embd, n_ff, S, ids, path=moe.PATH_GEMV)
    assert moe.last_stage_count() in (2, 3)     # gate/up, down with the sum, or the reduce behind it
    again = _ffn_case(E, k, T, n_embd, n_ff, S, ids, path=moe.PATH_GEMV)[0]
    assert torch.equal(got, again)


def test_narrow_rows_take_the_grouped_gemm():
    """Rows under 128 columns: the automatic choice is the grouped GEMM, the forced GEMV is refused."""
    ids = synth.draw_ids_uniform(3, 2, 4, 2)
    _mul_mat_id(4, 2, 2, 96, 40, 1, ids, moe.PATH_AUTO)
    assert moe.last_stage_count() == 2      # row ids with the quantization, GEMM
    with pytest.raises(moe.MoeError):
        _mul_mat_id(4, 2, 2, 96, 40, 1, ids, moe.PATH_GEMV)


@pytest.mark.parametrize("T", [40, 9])
def test_router_layer_and_graph(T):
    """Scored routing (one padding token) into the FFN on MXFP4 activations (grouped GEMM, and GEMV),
    with experts quantized here: eager, the no-allocation call and five replays of a captured graph
    give the same bytes."""
    E, k, n_embd, n_ff = 16, 4, 128, 160
    g = torch.Generator().manual_seed(3)
    mk = lambda *s: moe.Weights(*moe.moe_quantize_mxfp4((0.1 * torch.randn(s, generator=g)).cuda()))
    gate, up, down = mk(E, n_ff, n_embd), mk(E, n_ff, n_embd), mk(E, n_embd, n_ff)
    x = torch.randn((T, n_embd), generator=g).to(torch.bfloat16).cuda()
    logits = torch.randn((T, E), generator=g).cuda()
    logits[7] = -float("inf")
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    rw = torch.empty((T, k), device="cuda")
    out = torch.empty((T, n_embd), device="cuda")
    ws = torch.empty(moe.moe_ffn_fused_workspace_size(gate, None, T, k, act_quant=2), dtype=torch.uint8, device="cuda")

    def layer():
        moe.moe_router_scored(logits, k, score="sigmoid", n_group=4, topk_group=2, ids=ids, route_w=rw)
        moe.moe_ffn_fused(gate, up, down, x, ids, rw, out=out, workspace=ws, act_quant=2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.synchronize()
    ref = out.clone()
    assert (out[7] == 0).all() and torch.isfinite(out).all()
    hd = lambda w: ref64.decode(ref64.unpack(w.data.cpu().numpy()), w.scales.cpu().numpy())
    _check(out, *ref64.ffn(x.double().cpu().numpy(), hd(gate), hd(up), hd(down), ids.cpu().numpy(), rw.cpu().numpy()))
    noalloc = moe.moe_ffn_fused_noalloc(gate, up, down, x, ids, rw, act_quant=2)
    torch.cuda.synchronize()
    assert torch.equal(noalloc, ref)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        layer()
    for _ in range(5):
        out.fill_(float("nan"))
        ws.fill_(255)
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
        torch.randn(1 << 18, device="cuda").sum().item()
