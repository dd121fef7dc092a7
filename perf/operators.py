"""What the routing and MXFP4 operators are measured on: inputs, one pass, and the values it must give.

Four operators of a Mixture-of-Experts layer:
  route     router logits -> expert ids, routing weights and scores (softmax or sigmoid scores,
            a balance bias that only steers the choice, expert groups, top-k, renormalisation)
  grad      the gradient of the logits from the gradients of the routing weights and scores
  quant     rows -> MXFP4 (E2M1 codes, one E8M0 scale per 32 columns) and the values they stand for
  matmul    mul_mat_id of MXFP4 experts with activations quantised to MXFP4

With ``own`` false, ``run`` computes them in elementary torch operations; with ``own`` true it
calls the package. ``exact`` is the same from the definitions in 64 bits.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def _route(name, T, E, k, score, bias, groups, keep, group_top, renorm, scale, dtype, scores):
    return dict(name=name, op="route", T=T, E=E, k=k, score=score, bias=bias, groups=groups, keep=keep,
                group_top=group_top, renorm=renorm, scale=scale, dtype=dtype, scores=scores)


def _grad(name, T, E, k, score, renorm, scale, dtype, aux):
    return dict(name=name, op="grad", T=T, E=E, k=k, score=score, renorm=renorm, scale=scale, dtype=dtype, aux=aux)


def _quant(name, rows, K, dtype):
    return dict(name=name, op="quant", rows=rows, K=K, dtype=dtype)


def _matmul(name, T, E, k, N, K, weighted, per_slot, zipf, pad):
    return dict(name=name, op="matmul", T=T, E=E, k=k, N=N, K=K, weighted=weighted, per_slot=per_slot,
                zipf=zipf, pad=pad)


def listed():
    return [
        # one token of a decode step, DeepSeek-V3-shaped router: 256 experts in 8 groups
        _route("route_token", 1, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5, "float32", False),
        # the skewed prefill's router from bf16 logits, with the scores a balance loss reads
        _route("route_prefill_bf16", 4096, 128, 8, "softmax", False, 1, 1, 1, True, 1.0, "bfloat16", True),
        # a training step's tokens through the grouped, biased sigmoid router
        _route("route_train_grouped", 65536, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5, "float32", False),
        # router gradient of an odd batch, weights not renormalised, balance loss's gradient the same for all tokens
        _grad("grad_softmax_odd", 1021, 160, 6, "softmax", False, 16.0, "bfloat16", "row"),
        # router gradient of a training step with a gradient for every score
        _grad("grad_train_sigmoid", 65536, 256, 8, "sigmoid", True, 2.5, "float32", "full"),
        # activations of the GPT-OSS-shaped prefill
        _quant("quant_activations", 4096, 2880, "bfloat16"),
        # a whole stack of experts (32 x 2880 rows) from float32
        _quant("quant_experts_f32", 92160, 2880, "float32"),
        # one token's gate product, GPT-OSS-shaped
        _matmul("matmul_token", 1, 32, 4, 2880, 2880, False, False, 0.0, 0.0),
        # decode batch of 8: the weighted down product, each slot its own input row
        _matmul("matmul_decode_weighted", 8, 32, 4, 2880, 2880, True, True, 0.0, 0.0),
        # DeepSeek-Lite-shaped prompt of odd length, some of it padding
        _matmul("matmul_prompt_ragged", 509, 64, 6, 1408, 2048, False, False, 1.1, 0.05),
        # GPT-OSS-shaped prefill of 4096 tokens, weighted
        _matmul("matmul_prefill_weighted", 4096, 32, 4, 2880, 2880, True, False, 0.0, 0.0),
        # DeepSeek-V3-shaped widths, half of its experts
        _matmul("matmul_prefill_large", 4096, 128, 8, 2048, 7168, False, False, 0.0, 0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "grad", "quant", "matmul", "matmul"))
    if op in ("route", "grad"):
        groups = rng.choice((1, 1, 2, 4, 8))
        per = _log_int(rng, max(2, 8 // groups), 512 // groups)
        E = groups * per
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(16, keep * per))
        T = _log_int(rng, 1, min(65536, 65536 * 256 // E))
        score, renorm = rng.choice(("softmax", "sigmoid")), rng.random() < 0.6
        scale, dtype = rng.choice((1.0, 2.5, 16.0)), rng.choice(("float32", "bfloat16"))
        if op == "grad":
            c = _grad("", T, E, k, score, renorm, scale, dtype, rng.choice(("none", "row", "full")))
        else:
            c = _route("", T, E, k, score, rng.random() < 0.5, groups, keep, rng.choice((1, 2)), renorm, scale,
                       dtype, rng.random() < 0.5)
    elif op == "quant":
        K = 32 * _log_int(rng, 1, 256)
        c = _quant("", _log_int(rng, 1, 92160 * 2880 // K // 2), K, rng.choice(("float32", "bfloat16")))
    else:
        E = _log_int(rng, 4, 128)
        k = rng.randint(1, min(E, 8))
        N, K = _log_int(rng, 32, 4096), 32 * _log_int(rng, 2, 224)
        while E * N * K > 128 * 2048 * 7168:
            E = max(k, E // 2)
        most = 32768 * 2048 * 7168 // (N * K * k)
        c = _matmul("", _log_int(rng, 1, max(1, min(4096, most))), E, k, N, K, rng.random() < 0.5,
                    rng.random() < 0.5, rng.choice((0.0, 1.1)), rng.choice((0.0, 0.0, 0.1)))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _logits(case, g):
    """Router logits: a token's own part and a popularity that experts have for all tokens."""
    T, E = case["T"], case["E"]
    l = torch.randn((T, E), generator=g, device="cuda") * 1.5
    l += 0.7 * torch.randn((E,), generator=g, device="cuda")
    return l.to(getattr(torch, case["dtype"]))


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
    if case.get("zipf"):
        rank = torch.randperm(E, generator=g, device="cuda") + 1
        keys -= case["zipf"] * torch.log(rank.float())
    ids = torch.topk(keys, k, dim=1).indices.to(torch.int32)
    if case.get("pad"):
        ids[torch.rand((T,), generator=g, device="cuda") < case["pad"]] = -1
    return ids.contiguous()


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "route":
        s["logits"] = _logits(case, g)
        s["bias"] = 0.05 * torch.randn((case["E"],), generator=g, device="cuda") if case["bias"] else None
    elif case["op"] == "grad":
        T, E = case["T"], case["E"]
        s["logits"] = _logits(case, g)
        s["ids"] = torch.topk(s["logits"].float(), case["k"], dim=1).indices.to(torch.int32).contiguous()
        s["d_w"] = torch.randn((T, case["k"]), generator=g, device="cuda")
        shape = {"none": None, "row": (E,), "full": (T, E)}[case["aux"]]
        s["d_scores"] = None if shape is None else 0.1 * torch.randn(shape, generator=g, device="cuda")
    elif case["op"] == "quant":
        s["x"] = _activations(case["rows"], case["K"], case["dtype"], g)
    else:
        T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
        s["ids"] = _pick(case, g)
        rows = T * k if case["per_slot"] else T
        s["x"] = _activations(rows, K, "bfloat16", g)
        s["codes"] = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        s["scales"] = torch.randint(118, 122, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
        w = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), dim=1)
        s["route_w"] = w.contiguous() if case["weighted"] else None
        s["cap"] = max(1, int(torch.bincount(s["ids"].flatten() + 1, minlength=E + 1)[1:].max()))
    return s


# ------------------------------------------------------------------ one pass
def _run_own(s):
    import indirect_expert_matmul_amd as moe
    c = s["case"]
    if c["op"] == "route":
        return moe.moe_router_scored(s["logits"], c["k"], bias=s["bias"], score=c["score"], n_group=c["groups"],
                                     topk_group=c["keep"], group_top=c["group_top"], renorm=c["renorm"],
                                     scale=c["scale"], return_scores=c["scores"])
    if c["op"] == "grad":
        return moe.moe_router_scored_backward(s["logits"], s["ids"], s["d_w"], d_scores=s["d_scores"],
                                              score=c["score"], renorm=c["renorm"], scale=c["scale"])
    if c["op"] == "quant":
        codes, scales, values = moe.moe_quantize_mxfp4(s["x"], return_values=True)
        return codes, scales.view(torch.float8_e8m0fnu), values
    return moe.moe_mul_mat_id(moe.Weights(s["codes"], s["scales"]), s["x"], s["ids"], route_w=s["route_w"],
                              src1_rows_per_token=c["k"] if c["per_slot"] else 1, act_quant=2)


def _scores(l, score):
    return torch.softmax(l, dim=1) if score == "softmax" else torch.sigmoid(l)


def _route_plain(s):
    c = s["case"]
    T, E, G = c["T"], c["E"], c["groups"]
    p = _scores(s["logits"].double(), c["score"])     # 64 bits: two choices may be next to each other
    choice = p if s["bias"] is None else p + s["bias"].double()
    if G > 1:
        grouped = choice.view(T, G, E // G)
        top = torch.topk(grouped, min(c["group_top"], E // G), dim=2).values.sum(dim=2)
        kept = torch.sort(top, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        live = torch.zeros((T, G), dtype=torch.bool, device=choice.device).scatter_(1, kept, True)
        choice = grouped.masked_fill(~live[:, :, None], -math.inf).reshape(T, E)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    out = (ids.to(torch.int32), (w * c["scale"]).float())
    return out + (p.float(),) if c["scores"] else out


def _grad_plain(s):
    c = s["case"]
    p = _scores(s["logits"].float(), c["score"])
    ids = s["ids"].long()
    g = s["d_w"] * c["scale"]
    if c["renorm"]:
        picked = p.gather(1, ids)
        total = picked.sum(dim=1, keepdim=True)
        g = (g - (g * picked).sum(dim=1, keepdim=True) / total) / total
    d = torch.zeros_like(p).scatter_add_(1, ids, g)
    if s["d_scores"] is not None:
        d = d + s["d_scores"]
    d = p * (d - (d * p).sum(dim=1, keepdim=True)) if c["score"] == "softmax" else p * (1 - p) * d
    return d.to(s["logits"].dtype)


def _quantise(x):
    """Codes 0..15 and scale bytes of blocks of 32 (finite x): exponent of the largest magnitude less 2, codes to the
    nearest, ties to the even code, saturated at 6."""
    v = x.float().view(x.shape[0], -1, 32)
    top = v.abs().amax(dim=2)
    byte = ((top.view(torch.int32) >> 23) - 2).clamp_min(0)
    v = v * ((254 - byte) << 23).view(torch.float32)[:, :, None]
    a = v.abs()
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
            + 8 * torch.signbit(v))
    return code, byte


def _power(byte):
    """2^(byte - 127) for bytes 1 and up."""
    return (byte.int() << 23).view(torch.float32)


def _table(device):
    return torch.tensor(E2M1 + tuple(-v for v in E2M1), device=device)


def _decoded(code, byte):
    return (_table(code.device)[code] * _power(byte)[:, :, None]).view(code.shape[0], -1)


def _quant_plain(s):
    code, byte = _quantise(s["x"])
    flat = code.view(code.shape[0], -1)
    packed = (flat[:, ::2] | flat[:, 1::2] << 4).to(torch.uint8)
    return packed, byte.to(torch.uint8).view(torch.float8_e8m0fnu), _decoded(code, byte).to(s["x"].dtype)


def _matmul_plain(s):
    c = s["case"]
    T, E, k, N, K, cap = c["T"], c["E"], c["k"], c["N"], c["K"], s["cap"]
    x = _decoded(*_quantise(s["x"]))
    t = _table(x.device)
    pairs = torch.stack((t.repeat(16), t.repeat_interleave(16)), dim=1)
    w = pairs[s["codes"].view(-1).int()].view(E, N, K // 32, 32)
    w *= _power(s["scales"])[..., None]
    ids = s["ids"].flatten().long()
    e, entry = torch.sort(ids, stable=True)           # entries in expert order, padding first
    start = torch.searchsorted(e, torch.arange(E, device=e.device))
    at = torch.where(e >= 0, e * cap + torch.arange(T * k, device=e.device) - start[e.clamp_min(0)], E * cap)
    rows = torch.zeros((E * cap + 1, K), device=x.device)
    rows[at] = x[entry if c["per_slot"] else entry // k]
    y = torch.bmm(w.view(E, N, K), rows[:-1].view(E, cap, K).transpose(1, 2).contiguous())
    y = torch.cat((y.transpose(1, 2).reshape(E * cap, N), torch.zeros((1, N), device=x.device)))
    out = torch.empty((T * k, N), device=x.device)
    out[entry] = y[at] * (e >= 0)[:, None]
    out = out.view(T, k, N)
    return out if s["route_w"] is None else (out * s["route_w"][:, :, None]).sum(dim=1)


def run(state):
    if own:
        return _run_own(state)
    return {"route": _route_plain, "grad": _grad_plain, "quant": _quant_plain,
            "matmul": _matmul_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    width = 2 if case.get("dtype") == "bfloat16" else 4
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * (width + 4 * case["scores"]) + T * k * 8 + 4 * E * case["bias"],
                "flops": 8 * T * E + 2 * T * E * k}
    if op == "grad":
        T, E, k = case["T"], case["E"], case["k"]
        aux = {"none": 0, "row": 4 * E, "full": 4 * T * E}[case["aux"]]
        return {"bytes": 2 * T * E * width + T * k * 8 + aux, "flops": 10 * T * E}
    if op == "quant":
        n = case["rows"] * case["K"]
        return {"bytes": n * (2 * width + 17 / 32), "flops": 4 * n}
    T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
    touched = E * (1 - (1 - k / E) ** T)
    rows = T * (k if case["per_slot"] else 1)
    out = T * (1 if case["weighted"] else k) * N * 4
    return {"bytes": touched * N * K * 17 / 32 + rows * K * 2 + out + T * k * (8 if case["weighted"] else 4),
            "flops": 2.0 * T * k * N * K * (1 - case["pad"])}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_scores(case, l):
    if case["score"] == "softmax":
        z = torch.exp(l - l.max(dim=1, keepdim=True).values)
        return z / z.sum(dim=1, keepdim=True)
    return 1 / (1 + torch.exp(-l))


def _exact_route(case, s):
    T, E, G = case["T"], case["E"], case["groups"]
    p = _exact_scores(case, s["logits"].to(torch.float64))
    order = p.clone() if s["bias"] is None else p + s["bias"].to(torch.float64)
    best = order.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :case["group_top"]].sum(dim=2)
    for _ in range(G - case["keep"]):                 # drop the worst group, the last of equal ones
        worst = G - 1 - best.flip(1).argmin(dim=1)
        best.scatter_(1, worst[:, None], math.inf)
        order.view(T, G, E // G)[torch.arange(T, device=p.device), worst] = -math.inf
    w = torch.empty((T, case["k"]), dtype=torch.float64, device=p.device)
    for r in range(case["k"]):
        i = order.argmax(dim=1, keepdim=True)
        w[:, r:r + 1] = p.gather(1, i)
        order.scatter_(1, i, -math.inf)
    if case["renorm"]:
        w /= w.sum(dim=1, keepdim=True)
    return (None, w * case["scale"], p) if case["scores"] else (None, w * case["scale"])


def _exact_grad(case, s):
    l = s["logits"].to(torch.float64).requires_grad_(True)
    p = _exact_scores(case, l)
    w = torch.stack([p[torch.arange(case["T"], device=l.device), s["ids"][:, j].long()] for j in range(case["k"])], 1)
    if case["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    loss = (w * case["scale"] * s["d_w"].to(torch.float64)).sum()
    if s["d_scores"] is not None:
        loss = loss + (p * s["d_scores"].to(torch.float64)).sum()
    return torch.autograd.grad(loss, l)[0]


def _exact_power(e):
    """2^e in 64 bits, from its exponent field (pow() may be off by one in the last place, and so move a tie)."""
    return (e.long() + 1023 << 52).view(torch.float64)


def _exact_values(x):
    """(values, scales) of the nearest MXFP4 rows: steps of 1/2 below 2, of 1 below 4, of 2 up to 6."""
    v = x.to(torch.float64).view(x.shape[0], -1, 32)
    top = v.abs().amax(dim=2, keepdim=True)
    scale = _exact_power(torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp_min(-127))
    v = v / scale
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).to(torch.float64)
    v = (torch.round(v / step) * step).clamp(-6, 6) * scale
    return v.view(x.shape[0], -1), scale[:, :, 0]


def _exact_matmul(case, s):
    T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
    x, _ = _exact_values(s["x"])
    out = torch.zeros((T * k, N), dtype=torch.float64, device=x.device)
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=x.device)
    flat = s["ids"].flatten()
    for e in range(E):
        slots = torch.nonzero(flat == e).flatten()
        if not len(slots):
            continue
        b = s["codes"][e].long()
        w = torch.stack((grid[b & 15], grid[b >> 4]), dim=2).view(N, K // 32, 32)
        w = (w * _exact_power(s["scales"][e].long() - 127)[:, :, None]).view(N, K)
        out[slots] = x[slots if case["per_slot"] else slots // k] @ w.t()
    out = out.view(T, k, N)
    return out if s["route_w"] is None else (out * s["route_w"].to(torch.float64)[:, :, None]).sum(dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(case, s)
    if case["op"] == "grad":
        return _exact_grad(case, s)
    if case["op"] == "quant":
        values, scales = _exact_values(s["x"])
        return None, scales, values
    return _exact_matmul(case, s)
