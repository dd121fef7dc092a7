"""Scored routing, MXFP4 quantization and products of MXFP4 activations as programs use them: on
several streams, in several captured graphs, with used workspaces, and on tensors whose offsets pass
32 bits. Results are compared bit for bit with those of a single small call, which the other tests
compare with the float64 forms: a row's result depends on neither its position nor the batch."""
import pytest
import torch

import indirect_expert_matmul_amd as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _same(a, b):
    assert a.shape == b.shape and a.dtype == b.dtype
    kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    assert torch.equal(a.view(kind), b.view(kind))


def _codes(*shape):
    return torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda")


def _weights(E, N, K):
    return moe.Weights(_codes(E, N, K // 2), torch.randint(118, 122, (E, N, K // 32), dtype=torch.uint8, device="cuda"))


def _ids(T, E, k):
    return torch.rand((T, E), device="cuda").topk(k).indices.to(torch.int32)


class Layer:
    """Scored routing into the FFN on MXFP4 activations, all buffers its own."""

    def __init__(self, T, seed, E=16, k=4, n_embd=256, n_ff=160, shared=0):
        torch.manual_seed(seed)
        self.w = [_weights(E, n_ff, n_embd), _weights(E, n_ff, n_embd), _weights(E, n_embd, n_ff)]
        self.sh = [_weights(shared, n_ff, n_embd), _weights(shared, n_ff, n_embd),
                   _weights(shared, n_embd, n_ff)] if shared else None
        self.x = torch.randn((T, n_embd), device="cuda").to(torch.bfloat16)
        self.logits = torch.randn((T, E), device="cuda")
        self.logits[T // 2] = -float("inf")
        self.bias = 0.1 * torch.randn(E, device="cuda")
        self.ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
        self.rw = torch.empty((T, k), device="cuda")
        self.out = torch.empty((T, n_embd), device="cuda")
        need = moe.moe_ffn_fused_workspace_size(self.w[0], self.sh[0] if shared else None, T, k, act_quant=2)
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def run(self, workspace=True, stream=None):
        moe.moe_router_scored(self.logits, self.ids.shape[1], bias=self.bias, score="sigmoid", n_group=4,
                              topk_group=2, ids=self.ids, route_w=self.rw, stream=stream)
        moe.moe_ffn_fused(*self.w, self.x, self.ids, self.rw, shared=self.sh, out=self.out,
                          workspace=self.ws if workspace else None, act_quant=2, stream=stream)

    def clear(self):
        self.out.fill_(float("nan"))
        self.ids.fill_(-9)
        self.ws.fill_(255)


@pytest.mark.parametrize("T,shared", [(9, 0), (16, 2), (200, 1)])
def test_used_workspace_and_repeats(T, shared):
    a = Layer(T, 1, shared=shared)
    a.ws.zero_()
    a.run()
    torch.cuda.synchronize()
    ref = a.out.clone()
    assert torch.isfinite(ref).all()
    for i in range(10):
        a.clear()
        a.run()
        _same(a.out, ref)


@pytest.mark.parametrize("given", [False, True])
def test_two_streams_at_once(given):
    layers = [Layer(12, 1), Layer(300, 2, shared=1), Layer(64, 3)]
    refs = []
    for a in layers:
        a.run()
        torch.cuda.synchronize()
        refs.append(a.out.clone())
        a.clear()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(8):
        for a, st in zip(layers, streams):
            if given:      # the call's stream argument, with another one current
                a.run(workspace=False, stream=st)
            else:
                with torch.cuda.stream(st):
                    a.run(workspace=False)
    torch.cuda.synchronize()
    for a, ref in zip(layers, refs):
        _same(a.out, ref)


def test_two_graphs_replayed_in_turn():
    layers = [Layer(12, 1), Layer(300, 2, shared=1)]
    refs, graphs = [], []
    for a in layers:
        a.run()
        torch.cuda.synchronize()
        refs.append(a.out.clone())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            a.run()
        graphs.append(g)
    eager = Layer(40, 3)
    for i in range(5):
        for a in layers:
            a.clear()
        torch.cuda.synchronize()
        for g in graphs[::-1] if i % 2 else graphs:
            g.replay()
            eager.run(workspace=False)
        torch.cuda.synchronize()
        for a, ref in zip(layers, refs):
            _same(a.out, ref)


def test_graph_of_training_calls():
    """Routing, its gradient and fake quantization in one captured graph, five replays on new inputs."""
    T, E, k = 300, 64, 6
    logits = torch.empty((T, E), device="cuda")
    d_w = torch.empty((T, k), device="cuda")
    d_s = torch.empty(E, device="cuda")
    got = {}

    def step():
        ids, w, s = moe.moe_router_scored(logits, k, score="softmax", renorm=False, return_scores=True)
        grad = moe.moe_router_scored_backward(logits, ids, d_w, d_s, score="softmax", renorm=False)
        return [ids, w, s, grad, *moe.moe_quantize_mxfp4(logits, return_values=True)]
    gen = torch.Generator(device="cuda").manual_seed(5)

    def fill():
        for t in (logits, d_w, d_s):
            t.normal_(generator=gen)
    fill()
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(5):
        fill()
        g.replay()
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            _same(a, b)


@pytest.mark.parametrize("dtype,base,K,rep", [(torch.bfloat16, 4099, 2080, 520), (torch.float32, 1021, 4128, 1030)])
def test_quantize_past_32_bits(dtype, base, K, rep):
    assert base * K * rep > 2 ** 32
    x = (torch.randn((base, K), device="cuda") * torch.rand((base, 1), device="cuda") * 9).to(dtype)
    small = moe.moe_quantize_mxfp4(x, return_values=True)
    big = moe.moe_quantize_mxfp4(x.repeat(rep, 1), return_values=True)
    for a, b in zip(small, big):
        kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
        assert (b.view(kind).view(rep, base, -1) == a.view(kind)).all()


@pytest.mark.parametrize("E,k,dtype", [(512, 8, torch.float32), (1024, 8, torch.bfloat16), (1021, 20, torch.float32)])
def test_routing_and_gradient_past_32_bits(E, k, dtype):
    base, rep = 4099, 1023
    T = base * rep
    assert T < 2 ** 22 and 4 * T * E > 2 ** 32
    l = torch.randn((base, E), device="cuda").to(dtype)
    d_w, d_s = torch.randn((base, k), device="cuda"), torch.randn((base, E), device="cuda")
    kw = dict(score="sigmoid", renorm=True, scale=2.5)
    small = list(moe.moe_router_scored(l, k, return_scores=True, **kw))
    small.append(moe.moe_router_scored_backward(l, small[0], d_w, d_s, **kw))
    L = l.repeat(rep, 1)
    big = list(moe.moe_router_scored(L, k, return_scores=True, **kw))
    big.append(moe.moe_router_scored_backward(L, big[0], d_w.repeat(rep, 1), d_s.repeat(rep, 1), **kw))
    for a, b in zip(small, big):
        assert (b.view(rep, base, -1) == a).all()


@pytest.mark.parametrize("T,path", [(7, moe.PATH_GEMV), (7, moe.PATH_GEMM), (150, moe.PATH_GEMM)])
def test_expert_codes_past_32_bits(T, path):
    """9 GB of codes, of which the last two experts are used."""
    E, N, K = 67, 16384, 16416
    w = moe.Weights(_codes(E, N, K // 2), torch.full((E, N, K // 32), 120, dtype=torch.uint8, device="cuda"))
    assert w.data.numel() > 2 ** 33
    x = torch.randn((T, K), device="cuda").to(torch.bfloat16)
    ids = _ids(T, 2, 2)
    tail = moe.Weights(w.data[E - 2:], w.scales[E - 2:])
    a = moe.moe_mul_mat_id(tail, x, ids, act_quant=2, path=path)
    b = moe.moe_mul_mat_id(w, x, ids + (E - 2), act_quant=2, path=path)
    _same(a, b)
    assert a.abs().max() > 0


def test_activations_and_outputs_past_32_bits():
    """2.1 GB of gathered activation codes and 9.7 GB of output rows."""
    T, E, N, K, n = 264001, 3, 9216, 16416, 500
    w = _weights(E, N, K)
    x = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    x.normal_()
    ids = _ids(T, E, 1)
    out = moe.moe_mul_mat_id(w, x, ids, act_quant=2)
    assert out.numel() > 2 ** 31 and T * K // 2 > 2 ** 31
    for at in (0, T // 2, T - n):
        part = moe.moe_mul_mat_id(w, x[at:at + n], ids[at:at + n], act_quant=2, path=moe.PATH_GEMM)
        _same(out[at:at + n], part)


def test_ffn_intermediate_past_32_bits():
    """2.2 GB of codes of h."""
    T, k, E, n_embd, n_ff, n = 66003, 4, 5, 64, 16672, 300
    assert T * k * n_ff // 2 > 2 ** 31
    w = [_weights(E, n_ff, n_embd), _weights(E, n_ff, n_embd), _weights(E, n_embd, n_ff)]
    x = torch.randn((T, n_embd), device="cuda").to(torch.bfloat16)
    ids, rw = _ids(T, E, k), torch.rand((T, k), device="cuda")
    out = moe.moe_ffn_fused(*w, x, ids, rw, act_quant=2)
    for at in (0, T - n):
        part = moe.moe_ffn_fused(*w, x[at:at + n], ids[at:at + n], rw[at:at + n], act_quant=2, path=moe.PATH_GEMM)
        _same(out[at:at + n], part)
    assert torch.isfinite(out).all() and out.abs().max() > 0
