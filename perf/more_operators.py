"""The norm and the products in 8-bit floating point, in their plain form and as the library's calls, over the sizes they are used at.

``run(prepare(case, seed))`` is one pass through one operator. With ``own`` false it is computed by
elementary torch operations; with ``own`` true it makes the calls of trellis_coded_gemv_amd.binding
that a serving program makes.

  norm     rms_norm          residual addition, root-mean-square norm, and rows in 16 or 32 bits, in int8 with a scale for each row,
                             or in e4m3 with a scale for each 128 values
  quantize fp8_quantize      activation rows -> e4m3 rows with a scale for each 128 values
  gemm     fp8_gemm          e4m3 rows times an e4m3 layer with a scale for each block of 128 x 128
  experts  fp8_gemm_grouped  e4m3 rows times the experts that the tokens were routed to
"""
import math

import torch

own = False

BLOCK = 128
EPS = 1e-6
F8 = torch.float8_e4m3fn
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "int8": torch.int8, "fp8": F8}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "int8": 1, "fp8": 1, "none": 0}


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def listed():
    return [
        # one token between two trellis-coded layers, which give fp32 and take fp16: latency
        {"name": "norm_token", "op": "norm", "rows": 1, "n": 8192, "type": "f32", "residual": "f32", "weight": "f16", "out": "f16", "pad": 0},
        # a decode batch of odd size and width in front of an int8 layer
        {"name": "norm_batch_odd", "op": "norm", "rows": 61, "n": 5003, "type": "f16", "residual": "f16", "weight": "f16", "out": "int8", "pad": 5},
        # a long prompt in front of an e4m3 layer, at the benchmark's decoder width
        {"name": "norm_prompt", "op": "norm", "rows": 8192, "n": 8192, "type": "bf16", "residual": "bf16", "weight": "bf16", "out": "fp8", "pad": 0},
        # one token's activations at the benchmark's decoder width
        {"name": "quantize_token", "op": "quantize", "rows": 1, "n": 8192, "type": "f16", "pad": 0},
        # a prompt's activations in front of the 8B-shaped down projection
        {"name": "quantize_prompt", "op": "quantize", "rows": 4096, "n": 14336, "type": "bf16", "pad": 0},
        # one token through the benchmark's gate projection
        {"name": "gemm_token", "op": "gemm", "rows": 1, "m": 28672, "n": 8192, "out": "f32"},
        # a decode batch of odd size through the 8B-shaped down projection: few outputs, a long axis
        {"name": "gemm_batch_odd", "op": "gemm", "rows": 61, "m": 4096, "n": 14336, "out": "f32"},
        # a short prompt, ragged on every axis: part of a block at the end of both sides of the layer
        {"name": "gemm_ragged", "op": "gemm", "rows": 777, "m": 5003, "n": 4112, "out": "f16"},
        # a prompt through the benchmark's gate projection: the matrix cores' rate
        {"name": "gemm_prompt", "op": "gemm", "rows": 4096, "m": 28672, "n": 8192, "out": "bf16"},
        # one token's eight experts, gate and up in one layer each
        {"name": "experts_token", "op": "experts", "tokens": 1, "experts": 128, "top_k": 8, "m": 1536, "n": 2048, "per_pair": False, "out": "f32"},
        # the down products of a prompt's pairs, ragged groups
        {"name": "experts_down", "op": "experts", "tokens": 2000, "experts": 128, "top_k": 8, "m": 2048, "n": 768, "per_pair": True, "out": "f16"},
        # a prompt over all 128 experts, ragged groups
        {"name": "experts_prompt", "op": "experts", "tokens": 8192, "experts": 128, "top_k": 8, "m": 1536, "n": 2048, "per_pair": False, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "quantize", "gemm", "gemm", "experts", "experts"])
    kind = rng.choice(["f32", "f16", "bf16"])
    if op in ("norm", "quantize"):
        n = _log(rng, 64, 16384 if op == "norm" else 28672)
        n = n if rng.random() < 0.3 else (n + 15) // 16 * 16
        case = {"op": op, "rows": _log(rng, 1, min(8192, (1 << 26) // n)), "n": n, "type": kind}
        if op == "norm":
            case["residual"] = rng.choice(["none", kind, kind, rng.choice(["f32", "bf16"])])
            case["weight"] = rng.choice(["f32", kind])
            case["out"] = rng.choice(["f32", "f16", "bf16", "int8", "int8", "fp8", "fp8", "fp8"])
        case["pad"] = rng.choice([0, 0, 3, 64])
        return case
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


def _rows(rows, n, pad, seed, field, dtype):
    """Normal rows with a few outlying channels, as activations have them; pad > 0: a slice of wider rows."""
    x = torch.randn((rows, n + pad), generator=_gen(seed, field), device="cuda", dtype=torch.float32)
    x[:, :: 997] *= 12.0
    return x.to(dtype)[:, :n]


def _fp8(shape, seed, field):
    """e4m3 values of normally distributed weights or rows whose largest of 128 is about the type's largest."""
    return (torch.randn(shape, generator=_gen(seed, field), device="cuda", dtype=torch.float16) * 150.0).clamp_(-448, 448).to(F8)


def _scales(shape, seed, field):
    return torch.rand(shape, generator=_gen(seed, field), device="cuda", dtype=torch.float32) * 0.001 + 0.0002


def _ids(tokens, experts, top_k, seed):
    """Distinct experts of each token, some of them more popular than others."""
    liking = torch.randn(experts, generator=_gen(seed, 5), device="cuda") * 0.5
    return torch.topk(torch.randn((tokens, experts), generator=_gen(seed, 6), device="cuda") + liking, top_k, dim=1).indices.to(torch.int32)


def prepare(case, seed):
    op = case["op"]
    s = {"case": dict(case)}
    if op in ("norm", "quantize"):
        s["x"] = _rows(case["rows"], case["n"], case["pad"], seed, 0, DTYPES[case["type"]])
    if op == "norm":
        s["residual"] = None if case["residual"] == "none" else _rows(case["rows"], case["n"], 0, seed, 1, DTYPES[case["residual"]])
        s["weight"] = (torch.rand(case["n"], generator=_gen(seed, 2), device="cuda") + 0.5).to(DTYPES[case["weight"]])
    if op in ("gemm", "experts"):
        m, n = case["m"], case["n"]
        lead = () if op == "gemm" else (case["experts"],)
        s["wq"], s["sw"] = _fp8(lead + (m, n), seed, 0), _scales(lead + (_blocks(m), _blocks(n)), seed, 1)
        rows = case["rows"] if op == "gemm" else case["tokens"] * (case["top_k"] if case["per_pair"] else 1)
        s["xq"], s["sx"] = _fp8((rows, n), seed, 2), _scales((rows, _blocks(n)), seed, 3)
        if op == "experts":
            sel = _ids(case["tokens"], case["experts"], case["top_k"], seed).reshape(-1)
            s["order"] = torch.sort(sel, stable=True).indices.to(torch.int32)
            counts = torch.bincount(sel, minlength=case["experts"])
            s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        if own:  # the layer's descriptor and its workspace, which a program keeps from call to call
            from trellis_coded_gemv_amd import binding as tg
            if op == "gemm":
                s["layer"] = tg.Fp8Layer(s["wq"], s["sw"])
                s["ws"] = tg.fp8_workspace(s["layer"], rows)
            else:
                s["layer"] = tg.Fp8Experts(s["wq"], s["sw"])
    return s


def _to_blocks(v):
    """[..., n] -> [..., blocks, 128], zeros behind the last value."""
    n = v.shape[-1]
    return torch.nn.functional.pad(v, (0, _blocks(n) * BLOCK - n)).unflatten(-1, (-1, BLOCK))


def _round_e4m3(t):
    """The nearest multiple of the e4m3 step at each value of t (64 bits, |t| <= 448), halves to the even one."""
    step = torch.exp2((torch.frexp(t).exponent - 1).clamp(min=-6).double() - 3)
    return (torch.round(t / step) * step).to(F8)


def _plain_fp8(v, unit):
    """v's blocks as e4m3 steps (64 bits: a value next to the border of two steps goes to the nearer one) and their scales times unit."""
    b = _to_blocks(v)
    amax = b.abs().amax(-1, keepdim=True)
    q = _round_e4m3(b * 448.0 / amax).flatten(-2)[..., :v.shape[-1]]
    return {"q": q.contiguous(), "scale": (amax[..., 0] * unit / 448.0).float()}


def _plain_norm(s):
    c, out = s["case"], {}
    h = s["x"].float()
    if s["residual"] is not None:
        out["total"] = (h + s["residual"].float()).to(s["residual"].dtype)
        h = out["total"].float()
    unit = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    if c["out"] in ("int8", "fp8"):  # the steps do not depend on the norm, which scales a row as a whole
        v = h.double() * s["weight"].double()
        if c["out"] == "fp8":
            return out | _plain_fp8(v, unit)
        amax = v.abs().amax(1, keepdim=True)
        return out | {"q": torch.round(v * 127.0 / amax).to(torch.int8), "scale": (amax * unit / 127.0).float()[:, 0]}
    return out | {"y": (h * unit * s["weight"].float()).to(DTYPES[c["out"]])}


def _plain_quantize(s):
    return _plain_fp8(s["x"].double(), 1.0)


def _plain_product(xq, sx, wq, sw):
    x = xq.float() * sx.repeat_interleave(BLOCK, 1)[:, :xq.shape[1]]
    w = wq.float() * sw.repeat_interleave(BLOCK, 0)[:wq.shape[0]].repeat_interleave(BLOCK, 1)[:, :wq.shape[1]]
    return x @ w.t()


def _plain_gemm(s):
    return _plain_product(s["xq"], s["sx"], s["wq"], s["sw"]).to(DTYPES[s["case"]["out"]])


def _plain_experts(s):
    c = s["case"]
    pairs = s["order"].numel()
    y = torch.empty((pairs, c["m"]), device="cuda", dtype=DTYPES[c["out"]])
    at = s["offsets"].tolist()  # the plain form goes over the experts that have rows
    rows = s["xq"].view(torch.uint8)
    for e in range(c["experts"]):
        if at[e] < at[e + 1]:
            p = s["order"][at[e]:at[e + 1]].long()
            r = p if c["per_pair"] else p // c["top_k"]
            y[p] = _plain_product(rows[r].view(F8), s["sx"][r], s["wq"][e], s["sw"][e]).to(y.dtype)
    return y


def _own_norm(tg, s):
    c = s["case"]
    got = tg.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, out_dtype=DTYPES[c["out"]])
    names = (["q", "scale"] if c["out"] in ("int8", "fp8") else ["y"]) + ([] if s["residual"] is None else ["total"])
    return dict(zip(names, got if len(names) > 1 else [got]))


def _own_quantize(tg, s):
    q, scale = tg.fp8_quantize(s["x"])
    return {"q": q, "scale": scale}


def _own_gemm(tg, s):
    return tg.fp8_gemm(s["layer"], s["xq"], s["sx"], out_dtype=DTYPES[s["case"]["out"]], ws=s["ws"])


def _own_experts(tg, s):
    c = s["case"]
    return tg.fp8_gemm_grouped(s["layer"], s["xq"], s["sx"], s["offsets"], s["order"], pairs_per_row=1 if c["per_pair"] else c["top_k"],
                               out_dtype=DTYPES[c["out"]])


PLAIN = {"norm": _plain_norm, "quantize": _plain_quantize, "gemm": _plain_gemm, "experts": _plain_experts}
OWN = {"norm": _own_norm, "quantize": _own_quantize, "gemm": _own_gemm, "experts": _own_experts}


def run(state):
    if own:
        from trellis_coded_gemv_amd import binding as tg
        return OWN[state["case"]["op"]](tg, state)
    return PLAIN[state["case"]["op"]](state)


def work(case):
    op, n = case["op"], case["n"]
    if op == "norm":
        t = case["rows"]
        scales = 4 * t * {"int8": 1, "fp8": _blocks(n)}.get(case["out"], 0)
        return {"bytes": t * n * (SIZE[case["type"]] + 2 * SIZE[case["residual"]] + SIZE[case["out"]]) + n * SIZE[case["weight"]] + scales,
                "flops": 5 * t * n}
    if op == "quantize":
        t = case["rows"]
        return {"bytes": t * n * (SIZE[case["type"]] + 1) + 4 * t * _blocks(n), "flops": 3 * t * n}
    m = case["m"]
    layer = m * n + 4 * _blocks(m) * _blocks(n)
    if op == "gemm":
        t = case["rows"]
        return {"bytes": layer + t * (n + 4 * _blocks(n)) + t * m * SIZE[case["out"]], "flops": 2 * t * m * n}
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    pairs, rows = t * k, t * k if case["per_pair"] else t
    reached = e * (1.0 - (1.0 - k / e) ** t)  # experts that an even routing reaches
    return {"bytes": reached * layer + rows * (n + 4 * _blocks(n)) + 4 * pairs + 4 * (e + 1) + pairs * m * SIZE[case["out"]],
            "flops": 2 * pairs * m * n}


def _nearest(table, a, amax):
    """For each |value| a of a row whose largest is amax: the entry t of the rising table (even ones at even places) for which
    t / table[-1] is nearest to a / amax; ties go to the even place. By a search, corrected by exact differences."""
    top = table[-1]
    at = torch.searchsorted(table, a * top / amax, right=True).clamp(1, len(table) - 1)
    at = torch.where(a * top < table[at - 1] * amax, at - 1, at).clamp(min=1)
    below, above = a * top - table[at - 1] * amax, table[at] * amax - a * top
    up = (below > above) | ((below == above) & (at % 2 == 0))
    return torch.where(up, table[at], table[at - 1])


def _e4m3_values():
    """The type's finite values from 0 on: 8 below the smallest normal number's binade, then 8 to a binade, up to 448."""
    v = [i * 2.0 ** -9 for i in range(8)]
    v += [(8 + i) * 2.0 ** (e - 3) for e in range(-6, 9) for i in range(8)]
    return torch.tensor(v[:-1], dtype=torch.float64, device="cuda")


def _exact_steps(v, table, width):
    """Block by block of each row: the values that the steps stand for, and the largest of each block."""
    q, most = torch.zeros_like(v), []
    for b in range(0, v.shape[1], width):
        part = v[:, b:b + width]
        amax = part.abs().max(1).values
        q[:, b:b + width] = torch.sign(part) * _nearest(table, part.abs(), amax[:, None])
        most.append(amax)
    return q, torch.stack(most, 1)


def _exact_norm(c, s):
    h, out = s["x"].double(), {}
    if s["residual"] is not None:
        total = s["residual"].double() + h
        out["total"] = total
        if c["residual"] == "f32":  # the norm is that of the stored sum
            h = total.float().double()
        else:  # a sum of 16-bit values is rounded to 16 bits once: its rounding in 32 bits between changes nothing
            h = total.float().to(DTYPES[c["residual"]]).double()
    mean = torch.linalg.vector_norm(h, dim=1).square() / c["n"]
    v = h * s["weight"].double()
    if c["out"] in ("int8", "fp8"):
        table = _e4m3_values() if c["out"] == "fp8" else torch.arange(128, dtype=torch.float64, device="cuda")
        q, most = _exact_steps(v, table, BLOCK if c["out"] == "fp8" else c["n"])
        scale = most / table[-1] / torch.sqrt(mean + EPS)[:, None]
        return out | {"q": q, "scale": scale if c["out"] == "fp8" else scale[:, 0]}
    return out | {"y": v / torch.sqrt(mean + EPS)[:, None]}


def _exact_product(xq, sx, wq, sw):
    """Block by block of the inner axis: the products' sums, times the scales of the row and of the outputs' block."""
    y = torch.zeros(xq.shape[0], wq.shape[0], device="cuda", dtype=torch.float64)
    owner = torch.arange(wq.shape[0], device="cuda") // BLOCK
    for b in range(_blocks(xq.shape[1])):
        at = slice(b * BLOCK, (b + 1) * BLOCK)
        part = xq[:, at].double() @ wq[:, at].double().t()
        y += part.mul_(sx[:, b, None].double()).mul_(sw[owner, b].double())
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        return _exact_norm(case, s)
    if op == "quantize":
        q, most = _exact_steps(s["x"].double(), _e4m3_values(), BLOCK)
        return {"q": q, "scale": most / 448.0}
    if op == "gemm":
        return _exact_product(s["xq"], s["sx"], s["wq"], s["sw"])
    pairs = s["order"].numel()
    y = torch.zeros(pairs, case["m"], device="cuda", dtype=torch.float64)
    expert = torch.searchsorted(s["offsets"], torch.arange(pairs, device="cuda", dtype=torch.int32), right=True) - 1
    rows = s["xq"].float()
    for e in expert.unique().tolist():
        p = s["order"][expert == e].long()
        r = p if case["per_pair"] else torch.div(p, case["top_k"], rounding_mode="floor")
        y[p] = _exact_product(rows[r], s["sx"][r], s["wq"][e].float(), s["sw"][e])
    return y
