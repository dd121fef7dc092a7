"""What the 16-bit and 8-bit expert products are measured on: inputs, one pass, and the values it must give.

Operators of a Mixture-of-Experts layer, on tokens routed to k of E experts each:
  product   mul_mat_id of bfloat16 or float16 experts, per slot or as the weighted sum over a token's slots
  grads     its gradients: of the activations, of the experts and (weighted) of the routing weights
  rows      rows -> int8 codes with one float32 scale a row (d = max|x| / 127, codes to the nearest, ties to even)
  int8      mul_mat_id of int8 experts with a scale for each output row, activations as in ``rows``

With ``own`` false, ``run`` computes them in elementary torch operations; with ``own`` true it
calls the package. ``exact`` is the same from the definitions in 64 bits.
"""
import math

import torch

own = False


# ------------------------------------------------------------------ cases
def _slots(op, name, T, E, k, N, K, dtype, weighted, per_slot, zipf, pad, dw=""):
    return dict(name=name, op=op, T=T, E=E, k=k, N=N, K=K, dtype=dtype, weighted=weighted, per_slot=per_slot,
                zipf=zipf, pad=pad, dw=dw)


def _rows(name, rows, K, dtype):
    return dict(name=name, op="rows", rows=rows, K=K, dtype=dtype)


def listed():
    return [
        # one token's gate product, GPT-OSS-shaped
        _slots("product", "product_token", 1, 32, 4, 2880, 2880, "bfloat16", False, False, 0.0, 0.0),
        # decode batch of 8, DeepSeek-Lite-shaped weighted down product, each slot its own input row
        _slots("product", "product_decode_weighted", 8, 64, 6, 2048, 1408, "float16", True, True, 0.0, 0.0),
        # DeepSeek-Lite-shaped prompt of odd length with uneven experts, some of it padding
        _slots("product", "product_prompt_ragged", 509, 64, 6, 1408, 2048, "bfloat16", False, False, 1.1, 0.05),
        # DeepSeek-V3-shaped widths, half of its experts
        _slots("product", "product_prefill_large", 4096, 128, 8, 2048, 7168, "bfloat16", False, False, 0.0, 0.0),
        # gradients of a small batch with odd sizes, float16 with float32 gradients of the experts
        _slots("grads", "grads_small_odd", 61, 16, 4, 333, 520, "float16", False, True, 0.0, 0.1, "float32"),
        # a training step's gate product, DeepSeek-Lite-shaped, uneven experts, float32 gradients of the experts
        _slots("grads", "grads_train_uneven", 4096, 64, 6, 1408, 2048, "bfloat16", False, False, 1.1, 0.02, "float32"),
        # a training step's weighted down product, GPT-OSS-shaped, with the routing weights' gradient
        _slots("grads", "grads_train_weighted", 4096, 32, 4, 2880, 2880, "bfloat16", True, True, 0.0, 0.0, "bfloat16"),
        # activations of a prefill, DeepSeek-V3-shaped
        _rows("rows_activations", 4096, 7168, "bfloat16"),
        # a whole stack of experts (32 x 2880 rows) from float32
        _rows("rows_experts_f32", 92160, 2880, "float32"),
        # one token's gate product in 8 bits, GPT-OSS-shaped
        _slots("int8", "int8_token", 1, 32, 4, 2880, 2880, "bfloat16", False, False, 0.0, 0.0),
        # weighted product of an odd prompt in 8 bits, DeepSeek-Lite-shaped, some of it padding
        _slots("int8", "int8_prompt_weighted", 509, 64, 6, 2048, 1408, "bfloat16", True, True, 1.1, 0.05),
        # DeepSeek-V3-shaped widths in 8 bits, half of its experts
        _slots("int8", "int8_prefill_large", 4096, 128, 8, 2048, 7168, "bfloat16", False, False, 0.0, 0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("product", "product", "grads", "grads", "rows", "int8", "int8"))
    if op == "rows":
        K = rng.choice((1, 4, 16)) * _log_int(rng, 4, 512)
        c = _rows("", _log_int(rng, 1, 92160 * 2880 // K // 2), K, rng.choice(("float32", "bfloat16", "float16")))
    else:
        E = _log_int(rng, 4, 128)
        k = rng.randint(1, min(E, 8))
        N, K = _log_int(rng, 32, 4096), 16 * _log_int(rng, 2, 448)
        while E * N * K > 128 * 2048 * 7168 // (4 if op == "grads" else 1):
            E = max(k, E // 2)
            N = max(32, N // 2) if E == k else N
        most = 4096 * 4 * 2880 * 2880 // (N * K * k) if op == "grads" else 32768 * 2048 * 7168 // (N * K * k)
        T = _log_int(rng, 1, max(1, min(4096, most)))
        weighted = rng.random() < 0.5
        dtype = rng.choice(("bfloat16", "float16"))
        # a weighted gradient of the experts in their own type, the others in float32 too
        dw = "" if op != "grads" else dtype if weighted or rng.random() < 0.5 else "float32"
        c = _slots(op, "", T, E, k, N, K, dtype, weighted, rng.random() < 0.5, rng.choice((0.0, 1.1)),
                   rng.choice((0.0, 0.0, 0.1)), dw)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _activations(rows, K, dtype, g):
    """Rows of different size, with a few columns that stand out in all of them."""
    x = torch.randn((rows, K), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((rows, 1), generator=g, device="cuda"))
    loud = torch.rand((K,), generator=g, device="cuda") < 0.01
    return (x * torch.where(loud, 12.0, 1.0)).to(getattr(torch, dtype))


def _pick(case, g):
    """k distinct experts for each token, some tokens padding (id -1)."""
    T, E, k = case["T"], case["E"], case["k"]
    p = torch.rand((T, E), generator=g, device="cuda").clamp_min_(1e-20)
    keys = -torch.log(-torch.log(p))
    if case["zipf"]:
        rank = torch.randperm(E, generator=g, device="cuda") + 1
        keys -= case["zipf"] * torch.log(rank.float())
    ids = torch.topk(keys, k, dim=1).indices.to(torch.int32)
    if case["pad"]:
        ids[torch.rand((T,), generator=g, device="cuda") < case["pad"]] = -1
    return ids.contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "rows":
        s["x"] = _activations(case["rows"], case["K"], case["dtype"], g)
        return s
    T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
    dtype = getattr(torch, case["dtype"])
    s["ids"] = _pick(case, g)
    s["x"] = _activations(T * k if case["per_slot"] else T, K, case["dtype"], g)
    if case["op"] == "int8":
        s["w"] = torch.randint(-127, 128, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
        s["w_scale"] = (0.5 + torch.rand((E, N), generator=g, device="cuda")) * 4e-4
    else:
        s["w"] = torch.randn((E, N, K), generator=g, device="cuda", dtype=dtype) * 0.03
    rw = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), dim=1)
    s["route_w"] = rw.contiguous() if case["weighted"] else None
    if case["op"] == "grads":
        shape = (T, N) if case["weighted"] else (T, k, N)
        s["d_dst"] = (0.1 * torch.randn(shape, generator=g, device="cuda")).to(dtype)
    s["cap"] = max(1, int(torch.bincount(s["ids"].flatten() + 1, minlength=E + 1)[1:].max()))
    return s


# ------------------------------------------------------------------ one pass
def _run_own(s):
    import indirect_expert_matmul_amd as moe
    c = s["case"]
    if c["op"] == "rows":
        return moe.moe_quantize_rows(s["x"])
    B = c["k"] if c["per_slot"] else 1
    if c["op"] == "product":
        return moe.moe_mul_mat_id(moe.Weights(s["w"]), s["x"], s["ids"], route_w=s["route_w"], src1_rows_per_token=B)
    if c["op"] == "int8":
        return moe.moe_mul_mat_id(moe.Weights(s["w"], s["w_scale"]), s["x"], s["ids"], route_w=s["route_w"],
                                  src1_rows_per_token=B)
    grads = moe.moe_mul_mat_id_backward(moe.Weights(s["w"]), s["x"], s["ids"], s["d_dst"], route_w=s["route_w"],
                                        src1_rows_per_token=B, d_w_dtype=getattr(torch, c["dw"]))
    return grads if c["weighted"] else grads[:2]


def _quantise(x):
    """Int8 codes (as float32 numbers) and the scale of each row. Quotients of 64-bit numbers rounded to 32
    bits are the float32 quotients; a scalar divisor would become a product with its inverse."""
    v = x.double()
    d = (v.abs().amax(dim=1, keepdim=True) / 127.0).float()
    q = torch.where(d > 0, torch.round((v / d.double()).float()), 0.0).clamp_(-127, 127)
    return q, d


def _rows_plain(s):
    q, d = _quantise(s["x"])
    return q.to(torch.int8), d[:, 0]


class _Sorted:
    """The slots in expert order, each expert's rows padded to ``cap`` of a batched product."""

    def __init__(self, s):
        c = s["case"]
        self.E, self.k, self.cap, self.n = c["E"], c["k"], s["cap"], c["T"] * c["k"]
        e, self.slot = torch.sort(s["ids"].flatten().long(), stable=True)    # padding first
        start = torch.searchsorted(e, torch.arange(self.E, device=e.device))
        place = e * self.cap + torch.arange(self.n, device=e.device) - start[e.clamp_min(0)]
        self.valid = e >= 0
        self.at = torch.where(self.valid, place, self.E * self.cap)

    def rows(self, x, per_slot):
        """x's rows, one a slot or one a token, as [E][cap][K], zero where there is none."""
        r = torch.zeros((self.E * self.cap + 1, x.shape[-1]), device=x.device)
        r[self.at] = x[self.slot if per_slot else self.slot // self.k]
        return r[:-1].view(self.E, self.cap, -1)

    def slots(self, y):
        """[E][cap][N] back to slot order, zero rows for padding."""
        N = y.shape[2]
        y = torch.cat((y.reshape(self.E * self.cap, N), torch.zeros((1, N), device=y.device)))
        out = torch.empty((self.n, N), device=y.device)
        out[self.slot] = y[self.at] * self.valid[:, None]
        return out


def _product(s, x, w):
    """Per-slot rows [n][N] of float32 x and w."""
    o = _Sorted(s)
    return o.slots(torch.bmm(o.rows(x, s["case"]["per_slot"]), w.transpose(1, 2).contiguous()))


def _output(s, y):
    c = s["case"]
    y = y.view(c["T"], c["k"], c["N"])
    return y if s["route_w"] is None else (y * s["route_w"][:, :, None]).sum(dim=1)


def _product_plain(s):
    return _output(s, _product(s, s["x"].float(), s["w"].float()))


def _int8_plain(s):
    c = s["case"]
    q, d = _quantise(s["x"])
    y = _product(s, q, s["w"].float()) * (d if c["per_slot"] else d.repeat_interleave(c["k"], dim=0))
    ids = s["ids"].flatten().clamp_min(0).long()
    return _output(s, y * s["w_scale"][ids])


def _grads_plain(s):
    c = s["case"]
    T, k, N, K = (c[n] for n in ("T", "k", "N", "K"))
    o = _Sorted(s)
    x, w, dtype = s["x"].float(), s["w"].float(), s["x"].dtype
    dy = s["d_dst"].float()
    per_slot = s["route_w"] is None
    g = o.slots(torch.bmm(o.rows(dy.view(-1, N), per_slot), w))
    rw = None if per_slot else s["route_w"].view(T * k, 1)
    d_rw = None
    if not per_slot:
        d_rw = (g * (x if c["per_slot"] else x.repeat_interleave(k, dim=0))).sum(dim=1).view(T, k)
        g = g * rw
        dy = (s["route_w"][:, :, None] * dy[:, None, :])
    d_x = g if c["per_slot"] else g.view(T, k, K).sum(dim=1)
    d_w = torch.bmm(o.rows(dy.view(-1, N), True).transpose(1, 2).contiguous(), o.rows(x, c["per_slot"]))
    out = (d_x.to(dtype), d_w.to(getattr(torch, c["dw"])))
    return out if per_slot else out + (d_rw,)


def run(state):
    if own:
        return _run_own(state)
    return {"product": _product_plain, "grads": _grads_plain, "rows": _rows_plain,
            "int8": _int8_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    width = 4 if case["dtype"] == "float32" else 2
    if case["op"] == "rows":
        n = case["rows"] * case["K"]
        return {"bytes": n * (width + 1) + 4 * case["rows"], "flops": 4 * n}
    T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
    n = T * k * (1 - case["pad"])
    touched = E * (1 - (1 - k / E) ** T)
    rows = T * (k if case["per_slot"] else 1)
    maps = T * k * (8 if case["weighted"] else 4)
    if case["op"] == "grads":
        dy = T * (1 if case["weighted"] else k) * N * 2
        dw = E * N * K * (4 if case["dw"] == "float32" else 2)
        return {"bytes": touched * N * K * 2 + dy + 2 * rows * K * 2 + dw + maps + 4 * T * k * case["weighted"],
                "flops": 4.0 * n * N * K}
    out = T * (1 if case["weighted"] else k) * N * 4
    weights = touched * N * (K * 2 if case["op"] == "product" else K + 4)
    return {"bytes": weights + rows * K * 2 + out + maps, "flops": 2.0 * n * N * K}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_codes(x):
    """Codes and scales as 64-bit numbers. By definition the scale is a float32 number and the codes are
    decided by a float32 quotient (half of a row's largest value is a tie)."""
    v = x.to(torch.float64)
    d = torch.div(v.abs().max(dim=1).values, 127).to(torch.float32).to(torch.float64)
    q = torch.div(v, torch.where(d > 0, d, torch.ones_like(d)).unsqueeze(1)).to(torch.float32)
    return torch.round(q).to(torch.float64), d


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rows":
        return None, s["x"].to(torch.float64).abs().max(dim=1).values / 127
    T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
    flat = s["ids"].flatten()
    dev = flat.device
    rw = s["route_w"]
    x = s["x"]
    if case["op"] == "int8":
        q, d = _exact_codes(x)
        x = q * d[:, None]
    y = torch.zeros((T * k, N), dtype=torch.float64, device=dev)
    g = torch.zeros((T * k, K), dtype=torch.float64, device=dev)
    d_w = None
    if case["op"] == "grads":
        d_w = torch.zeros((E, N, K), dtype=torch.float64, device=dev)
    for e in range(E):
        slots = torch.nonzero(flat == e).flatten()
        if not len(slots):
            continue
        w = s["w"][e].to(torch.float64)
        if case["op"] == "int8":
            w = w * s["w_scale"][e].to(torch.float64)[:, None]
        xe = x[slots if case["per_slot"] else slots // k].to(torch.float64)
        if case["op"] == "grads":
            de = (s["d_dst"].view(-1, N)[slots // k if case["weighted"] else slots]).to(torch.float64)
            g[slots] = de @ w
            scaled = de if rw is None else de * rw.flatten()[slots].to(torch.float64)[:, None]
            d_w[e] = scaled.t().contiguous() @ xe
        else:
            y[slots] = xe @ w.t()
    if case["op"] != "grads":
        y = y.view(T, k, N)
        return y if rw is None else torch.einsum("tk,tkn->tn", rw.to(torch.float64), y)
    if rw is None:
        return (g if case["per_slot"] else g.view(T, k, K).sum(dim=1)), d_w
    weight = rw.to(torch.float64).flatten()[:, None]
    rows = x.to(torch.float64)[torch.arange(T * k, device=dev) // (1 if case["per_slot"] else k)]
    d_rw = torch.einsum("ik,ik->i", g, rows).view(T, k)
    d_x = g * weight
    return (d_x if case["per_slot"] else d_x.view(T, k, K).sum(dim=1)), d_w, d_rw
