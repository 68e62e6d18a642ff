"""The routing and 8-bit operators, in their plain form and as the library's calls, over the sizes they are used at.

``run(prepare(case, seed))`` is one pass through one operator. With ``own`` false it is computed by
elementary torch operations; with ``own`` true it makes the calls of trellis_coded_gemv_amd.binding
that a serving program makes.

  route    moe_route          router logits -> expert ids and weights of every token
  group    moe_group          expert ids -> (token, slot) pairs in expert order, offsets per expert
  quantize int8_quantize      activation rows -> 8-bit rows with a scale for each
  gemm     int8_gemm          8-bit rows times an 8-bit layer with a scale for each output channel
  experts  int8_gemm_grouped  8-bit rows times the experts that the tokens were routed to
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
NEG_INF = float("-inf")


def listed():
    return [
        # one token's router in the 128-expert block that the benchmark runs: latency
        {"name": "route_token", "op": "route", "tokens": 1, "experts": 128, "top_k": 8, "type": "f32", "sigmoid": False,
         "bias": False, "n_group": 1, "topk_group": 1, "group_top": 1, "renorm": True, "scale": 1.0, "pad": 0},
        # a decode batch of odd size, few experts, logits as a slice of a wider half-precision buffer
        {"name": "route_batch_odd", "op": "route", "tokens": 77, "experts": 60, "top_k": 4, "type": "bf16", "sigmoid": False,
         "bias": True, "n_group": 1, "topk_group": 1, "group_top": 1, "renorm": False, "scale": 1.0, "pad": 4},
        # a long prompt through a grouped router: sigmoid scores, a balancing bias, 4 of 8 groups
        {"name": "route_prompt_groups", "op": "route", "tokens": 8192, "experts": 256, "top_k": 8, "type": "f32", "sigmoid": True,
         "bias": True, "n_group": 8, "topk_group": 4, "group_top": 2, "renorm": True, "scale": 2.5, "pad": 0},
        # the pairs of the benchmark's 64 tokens, top 8 of 128
        {"name": "group_batch", "op": "group", "tokens": 64, "experts": 128, "top_k": 8},
        # the pairs of a long prompt
        {"name": "group_prompt", "op": "group", "tokens": 16384, "experts": 256, "top_k": 8},
        # one token's activations at the benchmark's decoder width
        {"name": "quantize_token", "op": "quantize", "rows": 1, "n": 8192, "type": "f16", "pad": 0},
        # a prompt's activations in front of the 8B-shaped down projection
        {"name": "quantize_prompt", "op": "quantize", "rows": 4096, "n": 14336, "type": "bf16", "pad": 0},
        # one token through the benchmark's gate projection
        {"name": "gemm_token", "op": "gemm", "rows": 1, "m": 28672, "n": 8192, "out": "f32"},
        # a decode batch of odd size through the 8B-shaped down projection: few outputs, a long axis
        {"name": "gemm_batch_odd", "op": "gemm", "rows": 61, "m": 4096, "n": 14336, "out": "f32"},
        # a prompt through the benchmark's gate projection: the matrix cores' rate
        {"name": "gemm_prompt", "op": "gemm", "rows": 4096, "m": 28672, "n": 8192, "out": "bf16"},
        # one token's eight experts, gate and up in one layer each
        {"name": "experts_token", "op": "experts", "tokens": 1, "experts": 128, "top_k": 8, "m": 1536, "n": 2048, "per_pair": False, "out": "f32"},
        # a prompt over all 128 experts, ragged groups
        {"name": "experts_prompt", "op": "experts", "tokens": 8192, "experts": 128, "top_k": 8, "m": 1536, "n": 2048, "per_pair": False, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "group", "quantize", "gemm", "gemm", "experts", "experts"])
    kind = rng.choice(["f32", "f16", "bf16"])
    if op == "route":
        n_group = rng.choice([1, 1, 2, 4, 8])
        experts = n_group * _log(rng, max(2, 8 // n_group), 512 // n_group)
        topk_group = rng.randint(1, n_group)
        return {"op": op, "tokens": _log(rng, 1, 8192), "experts": experts,
                "top_k": rng.randint(1, min(16, experts // n_group * topk_group)), "type": kind,
                "sigmoid": rng.random() < 0.5, "bias": rng.random() < 0.5, "n_group": n_group, "topk_group": topk_group,
                "group_top": rng.choice([1, 2]), "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5]),
                "pad": rng.choice([0, 0, 1, 8])}
    if op == "group":
        experts = _log(rng, 8, 512)
        return {"op": op, "tokens": _log(rng, 1, 16384), "experts": experts, "top_k": rng.randint(1, 8)}
    if op == "quantize":
        n = _log(rng, 64, 28672)
        n = n if rng.random() < 0.3 else (n + 15) // 16 * 16
        return {"op": op, "rows": _log(rng, 1, min(8192, (1 << 26) // n)), "n": n, "type": kind, "pad": rng.choice([0, 0, 3, 64])}
    if op == "gemm":
        m, n = _log(rng, 128, 28672), (_log(rng, 128, 28672) + 15) // 16 * 16
        m = m if rng.random() < 0.4 else (m + 127) // 128 * 128
        rows = _log(rng, 1, max(1, min(8192, 9 * 10 ** 11 // (m * n))))
        return {"op": op, "rows": rows, "m": m, "n": n, "out": kind}
    experts = _log(rng, 8, 128)
    m, n = (_log(rng, 256, 4096) + 15) // 16 * 16, (_log(rng, 256, 4096) + 15) // 16 * 16
    top_k = rng.randint(1, 8)
    tokens = _log(rng, 1, max(1, min(8192, (1 << 27) // (top_k * max(m, n)))))
    return {"op": op, "tokens": tokens, "experts": min(experts, max(8, (1 << 29) // (m * n))), "top_k": top_k, "m": m, "n": n,
            "per_pair": rng.random() < 0.5, "out": kind}


def _gen(seed, field):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 16 + field)
    return g


def _normal(shape, seed, field, dtype=torch.float32):
    return torch.randn(shape, generator=_gen(seed, field), device="cuda", dtype=torch.float32).to(dtype)


def _rows(rows, n, pad, seed, field, dtype):
    """Normal rows with a few outlying channels, as activations have them; pad > 0: a slice of wider rows."""
    x = torch.randn((rows, n + pad), generator=_gen(seed, field), device="cuda", dtype=torch.float32)
    x[:, :: 997] *= 12.0
    return x.to(dtype)[:, :n]


def _int8(shape, seed, field):
    """8-bit values of normally distributed weights or rows, three standard deviations inside the range."""
    return (torch.randn(shape, generator=_gen(seed, field), device="cuda", dtype=torch.float16) * 40.0).round_().clamp_(-127, 127).to(torch.int8)


def _scales(shape, seed, field):
    return torch.rand(shape, generator=_gen(seed, field), device="cuda", dtype=torch.float32) * 0.01 + 0.002


def _ids(tokens, experts, top_k, seed):
    """Distinct experts of each token, some of them more popular than others."""
    liking = _normal((experts,), seed, 5) * 0.5
    return torch.topk(_normal((tokens, experts), seed, 6) + liking, top_k, dim=1).indices.to(torch.int32)


def prepare(case, seed):
    op = case["op"]
    s = {"case": dict(case)}
    if op == "route":
        wide = _normal((case["tokens"], case["experts"] + case["pad"]), seed, 0, DTYPES[case["type"]])
        s["logits"] = wide[:, :case["experts"]]
        s["bias"] = _normal((case["experts"],), seed, 1) * 0.05 if case["bias"] else None
    elif op == "group":
        s["sel"] = _ids(case["tokens"], case["experts"], case["top_k"], seed)
    elif op == "quantize":
        s["x"] = _rows(case["rows"], case["n"], case["pad"], seed, 0, DTYPES[case["type"]])
    else:
        shape = (case["m"], case["n"]) if op == "gemm" else (case["experts"], case["m"], case["n"])
        s["wq"], s["sw"] = _int8(shape, seed, 0), _scales(shape[:-1], seed, 1)
        rows = case["rows"] if op == "gemm" else case["tokens"] * (case["top_k"] if case["per_pair"] else 1)
        s["xq"], s["sx"] = _int8((rows, case["n"]), seed, 2), _scales((rows,), seed, 3)
        if op == "experts":
            sel = _ids(case["tokens"], case["experts"], case["top_k"], seed).reshape(-1)
            s["order"] = torch.sort(sel, stable=True).indices.to(torch.int32)
            counts = torch.bincount(sel, minlength=case["experts"])
            s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        if own:  # the layer's descriptor and its workspace, which a program keeps from call to call
            from trellis_coded_gemv_amd import binding as tg
            if op == "gemm":
                s["layer"] = tg.Int8Layer(s["wq"], s["sw"])
                s["ws"] = tg.int8_workspace(s["layer"], rows)
            else:
                s["layer"] = tg.Int8Experts(s["wq"], s["sw"])
    return s


def _plain_route(s):
    c = s["case"]
    experts, groups, k = c["experts"], c["n_group"], c["top_k"]
    l = s["logits"].double()  # 64 bits: scores decide which experts are taken, and some lie close together
    if c["sigmoid"]:
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        e = torch.exp(l - l.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    ranked = score if s["bias"] is None else score + s["bias"].double()
    key = l if s["bias"] is None else ranked
    if groups > 1:
        best = torch.sort(ranked.view(-1, groups, experts // groups), dim=2, descending=True).values
        value = best[:, :, :c["group_top"]].sum(2)
        kept = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        keep = torch.zeros_like(value).scatter_(1, kept, 1.0) > 0
        key = torch.where(keep.repeat_interleave(experts // groups, 1), key, NEG_INF)
    sel = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, sel)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"sel": sel.to(torch.int32), "weights": (w * c["scale"]).float()}


def _plain_group(s):
    sel = s["sel"].reshape(-1)
    experts = torch.arange(s["case"]["experts"] + 1, device=sel.device, dtype=torch.int32)
    ordered, order = torch.sort(sel, stable=True)
    return {"offsets": torch.searchsorted(ordered, experts).to(torch.int32), "order": order.to(torch.int32)}


def _plain_quantize(s):
    x = s["x"].double()  # 64 bits: a value next to the border of two steps goes to the nearer one
    amax = x.abs().amax(1, keepdim=True)
    # q is the operator's whole numbers and has to be equal; scale is what one step of its row stands for
    return {"q": torch.round(x * 127.0 / amax).to(torch.int8), "scale": (amax[:, 0] / 127.0).float()}


def _plain_gemm(s):
    y = s["xq"].float() @ s["wq"].float().t()
    return (y * s["sx"][:, None] * s["sw"]).to(DTYPES[s["case"]["out"]])


def _plain_experts(s):
    c = s["case"]
    pairs = s["order"].numel()
    y = torch.empty((pairs, c["m"]), device="cuda", dtype=DTYPES[c["out"]])
    at = s["offsets"].tolist()  # the plain form goes over the experts that have rows
    for e in range(c["experts"]):
        if at[e] < at[e + 1]:
            p = s["order"][at[e]:at[e + 1]].long()
            r = p if c["per_pair"] else p // c["top_k"]
            y[p] = (s["xq"][r].float() @ s["wq"][e].float().t() * s["sx"][r][:, None] * s["sw"][e]).to(y.dtype)
    return y


def _own_route(tg, s):
    c = s["case"]
    sel, w = tg.moe_route(s["logits"], c["top_k"], bias=s["bias"], sigmoid=c["sigmoid"], n_group=c["n_group"], topk_group=c["topk_group"],
                          group_top=c["group_top"], renormalize=c["renorm"], scale=c["scale"])
    return {"sel": sel, "weights": w}


def _own_group(tg, s):
    offsets, order = tg.moe_group(s["sel"], s["case"]["experts"])
    return {"offsets": offsets, "order": order}


def _own_quantize(tg, s):
    q, scale = tg.int8_quantize(s["x"])
    return {"q": q, "scale": scale}


def _own_gemm(tg, s):
    return tg.int8_gemm(s["layer"], s["xq"], s["sx"], out_dtype=DTYPES[s["case"]["out"]], ws=s["ws"])


def _own_experts(tg, s):
    c = s["case"]
    return tg.int8_gemm_grouped(s["layer"], s["xq"], s["sx"], s["offsets"], s["order"], pairs_per_row=1 if c["per_pair"] else c["top_k"],
                                out_dtype=DTYPES[c["out"]])


PLAIN = {"route": _plain_route, "group": _plain_group, "quantize": _plain_quantize, "gemm": _plain_gemm, "experts": _plain_experts}
OWN = {"route": _own_route, "group": _own_group, "quantize": _own_quantize, "gemm": _own_gemm, "experts": _own_experts}


def run(state):
    if own:
        from trellis_coded_gemv_amd import binding as tg
        return OWN[state["case"]["op"]](tg, state)
    return PLAIN[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        return {"bytes": t * e * SIZE[case["type"]] + (4 * e if case["bias"] else 0) + 8 * t * k, "flops": 4 * t * e}
    if op == "group":
        return {"bytes": 8 * case["tokens"] * case["top_k"] + 4 * (case["experts"] + 1), "flops": 0}
    if op == "quantize":
        t, n = case["rows"], case["n"]
        return {"bytes": t * n * (SIZE[case["type"]] + 1) + 4 * t, "flops": 3 * t * n}
    m, n = case["m"], case["n"]
    if op == "gemm":
        t = case["rows"]
        return {"bytes": m * n + t * n + 4 * (m + t) + t * m * SIZE[case["out"]], "flops": 2 * t * m * n}
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    pairs, rows = t * k, t * k if case["per_pair"] else t
    reached = e * (1.0 - (1.0 - k / e) ** t)  # experts that an even routing reaches
    return {"bytes": reached * (m * n + 4 * m) + rows * (n + 4) + 4 * pairs + 4 * (e + 1) + pairs * m * SIZE[case["out"]], "flops": 2 * pairs * m * n}


def _exact_route(c, s):
    """Expert by expert: one is taken if fewer than top_k others stand before it."""
    l = s["logits"].double().cpu()
    tokens, experts = l.shape
    if c["sigmoid"]:
        score = torch.sigmoid(l)
    else:
        score = torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
    with_bias = score if s["bias"] is None else score + s["bias"].double().cpu()
    key = (l if s["bias"] is None else with_bias).clone()
    if c["n_group"] > 1:
        size = experts // c["n_group"]
        value = torch.stack([torch.topk(with_bias[:, g * size:(g + 1) * size], min(c["group_top"], size), dim=1).values.sum(1)
                             for g in range(c["n_group"])], 1)
        for g in range(c["n_group"]):
            before = (value > value[:, g:g + 1]).sum(1) + (value[:, :g] == value[:, g:g + 1]).sum(1)
            key[before >= c["topk_group"], g * size:(g + 1) * size] = NEG_INF
    sel = torch.zeros(tokens, c["top_k"], dtype=torch.int64)
    w = torch.zeros(tokens, c["top_k"], dtype=torch.float64)
    every = torch.arange(tokens)
    for i in range(c["top_k"]):
        top = key.amax(1, keepdim=True)
        at = (key == top).to(torch.int8).argmax(1)  # the first of equal ones
        sel[:, i], w[:, i] = at, score[every, at]
        key[every, at] = NEG_INF
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"sel": sel, "weights": w * c["scale"]}


def _exact_quantize(s):
    """127 |x| / amax by its whole part and the exact rest."""
    x = s["x"].double()
    amax = x.abs().amax(1, keepdim=True)
    a = 254.0 * x.abs()
    whole = torch.floor(a / (2.0 * amax))
    rest = a - 2.0 * amax * whole
    up = (rest > amax) | ((rest == amax) & (whole.remainder(2.0) == 1.0))
    return {"q": ((whole + up.double()) * torch.sign(x)).to(torch.int8), "scale": amax[:, 0] / 127.0}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(case, s)
    if op == "group":
        return None  # whole numbers only
    if op == "quantize":
        return _exact_quantize(s)
    w = s["wq"].reshape(-1, case["m"], case["n"])
    scaled = s["xq"].double() * s["sx"].double()[:, None]
    if op == "gemm":
        return (scaled @ w[0].double().t()) * s["sw"].double()
    pairs = s["order"].numel()
    y = torch.zeros(pairs, case["m"], device="cuda", dtype=torch.float64)
    expert = torch.searchsorted(s["offsets"], torch.arange(pairs, device="cuda", dtype=torch.int32), right=True) - 1
    for e in expert.unique().tolist():
        p = s["order"][expert == e].long()
        r = p if case["per_pair"] else torch.div(p, case["top_k"], rounding_mode="floor")
        y[p] = (scaled[r] @ w[e].double().t()) * s["sw"][e].double()
    return y
