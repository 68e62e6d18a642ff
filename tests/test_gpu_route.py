"""moe_route and moe_group on the GPU against the float64 oracle: ids equal, weights within their one rounding."""
import numpy as np
import pytest

from gpu_common import device, say
from oracle import route as oracle
from trellis_coded_gemv_amd import binding as tg

pytestmark = pytest.mark.gpu

# A weight is formed in binary64 (a few roundings of 2^-53, far below) and rounded to binary32 once: half a step,
# 2^-24 relative; 1e-6 of that covers the binary64 part.
W_TOL = 2.0 ** -24 * (1 + 1e-6)

CASES = [  # tokens, experts, top_k, type, options
    (1, 128, 8, "float32", {}),
    (1, 1, 1, "float32", {}),
    (2, 5, 5, "float32", dict(renormalize=False, scale=2.5)),
    (77, 60, 4, "bfloat16", dict(bias=True, renormalize=False)),
    (33, 64, 64, "float32", {}),
    (9, 65, 3, "float16", dict(sigmoid=True)),
    (40, 128, 8, "bfloat16", {}),
    (40, 200, 16, "float32", dict(sigmoid=True, bias=True, scale=0.5)),
    (70, 256, 8, "float32", dict(sigmoid=True, bias=True, n_group=8, topk_group=4, group_top=2, scale=2.5)),
    (70, 256, 8, "bfloat16", dict(n_group=8, topk_group=3, group_top=1)),
    (31, 256, 6, "float16", dict(bias=True, n_group=64, topk_group=2, group_top=2)),
    (31, 24, 6, "float32", dict(n_group=24, topk_group=6, group_top=2)),
    (17, 512, 10, "float32", dict(sigmoid=True, n_group=4, topk_group=1, group_top=2)),
    (5, 1000, 12, "bfloat16", dict(bias=True)),
    (6, 1024, 64, "float32", dict(sigmoid=True, bias=True)),
]


def _check(torch, dev, logits, top_k, opts, pad=0, dtype="float32"):
    """logits: float32 array already representable in dtype."""
    kw = dict(opts)
    bias = kw.pop("bias", None)
    wide = np.full((logits.shape[0], logits.shape[1] + pad), np.nan, np.float32)   # what lies between rows is never read
    wide[:, :logits.shape[1]] = logits
    t = torch.from_numpy(wide).to(dev).to(getattr(torch, dtype))[:, :logits.shape[1]]
    T = logits.shape[0]
    sel = torch.full((T + 2, top_k), 77, dtype=torch.int32, device=dev)
    w = torch.full((T + 2, top_k), 77.0, device=dev)
    tg.moe_route(t, top_k, bias=None if bias is None else torch.from_numpy(bias).to(dev), sel=sel[1:T + 1], weights=w[1:T + 1], **kw)
    torch.cuda.synchronize()
    sel, w = sel.cpu().numpy(), w.cpu().numpy()
    assert (sel[0] == 77).all() and (sel[-1] == 77).all() and (w[0] == 77).all() and (w[-1] == 77).all()
    ids, ref = oracle.route(logits, top_k, bias=bias, **kw)
    assert np.array_equal(sel[1:-1], ids)
    got = w[1:-1].astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    assert np.all(np.abs(got[ok] - ref[ok]) <= W_TOL * np.abs(ref[ok]) + 2.0 ** -150)


@pytest.mark.parametrize("tokens,experts,top_k,dtype,opts", CASES)
def test_route_matches_oracle(tokens, experts, top_k, dtype, opts):
    dev = device()
    import torch
    say("route", tokens, experts, top_k, dtype, opts)
    rng = np.random.default_rng(tokens * 1000 + experts)
    l = torch.from_numpy((rng.normal(size=(tokens, experts)) * 2).astype(np.float32)).to(getattr(torch, dtype)).float().numpy()
    opts = dict(opts)
    if opts.get("bias"):
        opts["bias"] = (rng.normal(size=experts) * 0.1).astype(np.float32)
    _check(torch, dev, l, top_k, opts, pad=tokens % 3, dtype=dtype)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("experts", [40, 128, 192, 256, 384, 512, 1008, 1024])
@pytest.mark.parametrize("shift,pad", [(0, 0), (0, 16), (1, 15), (0, 1), (8, 0)])
def test_rows_read_at_once_or_one_by_one(dtype, experts, shift, pad):
    """Rows at every alignment, aligned and shifted biases; what lies beside the rows is never used."""
    dev = device()
    import torch
    say("route rows", dtype, experts, shift, pad)
    rng = np.random.default_rng(experts + shift * 7 + pad)
    T, top_k, ld = 5, 6, experts + pad
    l = torch.from_numpy((rng.normal(size=(T, experts)) * 2).astype(np.float32)).to(getattr(torch, dtype))
    flat = torch.full((shift + T * ld,), float("nan"), dtype=l.dtype, device=dev)
    view = flat[shift:].as_strided((T, experts), (ld, 1))
    view.copy_(l)
    bias = rng.normal(size=experts).astype(np.float32) * 0.1
    wide_bias = torch.full((shift + experts,), float("nan"), device=dev)
    wide_bias[shift:].copy_(torch.from_numpy(bias))
    for b, b_np in [(None, None), (wide_bias[shift:], bias)]:
        sel, w = tg.moe_route(view, top_k, bias=b, sigmoid=True)
        ids, ref = oracle.route(l.float().numpy(), top_k, bias=b_np, sigmoid=True)
        assert np.array_equal(sel.cpu().numpy(), ids)
        assert np.all(np.abs(w.cpu().numpy().astype(np.float64) - ref) <= W_TOL * ref)


@pytest.mark.parametrize("opts", [{}, dict(sigmoid=True), dict(n_group=8, topk_group=3, group_top=2), dict(sigmoid=True, zero_bias=True)])
def test_equal_logits_go_to_the_lowest_index(opts):
    dev = device()
    import torch
    say("route ties", opts)
    rng = np.random.default_rng(11)
    l = rng.integers(-2, 3, size=(64, 128)).astype(np.float32)     # five values over 128 experts
    opts = dict(opts)
    if opts.pop("zero_bias", False):
        opts["bias"] = np.zeros(128, np.float32)
    _check(torch, dev, l, 8, opts)


@pytest.mark.parametrize("experts", [33, 64, 100, 256, 512, 1000])
@pytest.mark.parametrize("opts", [{}, dict(sigmoid=True, zero_bias=True), dict(renormalize=False)])
def test_equal_logits_in_one_lane(experts, opts):
    """Few values, masked experts between them, and more of the largest than slots: neighbours with equal keys keep their order
    however many experts a lane holds."""
    dev = device()
    import torch
    say("route ties in a lane", experts, opts)
    rng = np.random.default_rng(experts)
    l = rng.integers(0, 3, size=(48, experts)).astype(np.float32)
    l[rng.random(l.shape) < 0.2] = -np.inf
    l[0] = 1.0
    l[1, : experts // 2] = -np.inf
    opts = dict(opts)
    if opts.pop("zero_bias", False):
        opts["bias"] = np.zeros(experts, np.float32)
    _check(torch, dev, l, 32, opts)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_unavailable_experts_and_tokens_without_order(sigmoid):
    """Masked logits (-inf, also whole rows and whole groups), the type's lowest value, NaN and +inf in single tokens."""
    dev = device()
    import torch
    rng = np.random.default_rng(12)
    inf = np.inf
    l = rng.normal(size=(12, 32)).astype(np.float32)
    l[0, :] = -inf
    l[1, 1:] = -inf
    l[2, ::2] = -inf
    l[3, 5] = np.nan
    l[4, 9] = inf
    l[5, :] = np.finfo(np.float32).min
    l[6, :8] = -inf
    l[7, 1:8] = -inf
    l[8, :] = np.finfo(np.float32).max
    l[9, 3] = 60000.0
    l[10, :30] = -inf
    for opts in (dict(sigmoid=sigmoid), dict(sigmoid=sigmoid, n_group=4, topk_group=2, group_top=2),
                 dict(sigmoid=sigmoid, renormalize=False, bias=np.where(np.arange(32) % 5 == 0, -inf, 0.01 * np.arange(32)).astype(np.float32)),
                 dict(sigmoid=sigmoid, bias=np.where(np.arange(32) == 4, np.nan, 0.0).astype(np.float32)),
                 dict(sigmoid=sigmoid, bias=np.where(np.arange(32) == 4, inf, 0.0).astype(np.float32))):
        say("route masks", sorted(opts))
        _check(torch, dev, l, 6, opts)


def test_close_scores_are_decided_in_64_bits():
    """Sigmoid scores plus biases that differ by less than a binary32 step: the larger one is taken all the same."""
    dev = device()
    import torch
    say("route close scores")
    rng = np.random.default_rng(13)
    base = rng.normal(size=(50, 1)).astype(np.float32)
    l = (base + np.float32(1e-7) * rng.integers(-3, 4, size=(50, 64))).astype(np.float32)
    bias = (np.float32(0.25) + np.float32(2.0 ** -26) * rng.integers(0, 4, size=64)).astype(np.float32)
    _check(torch, dev, l, 8, dict(sigmoid=True, bias=bias))
    _check(torch, dev, l, 8, dict(bias=bias, n_group=8, topk_group=4, group_top=2, sigmoid=True))


@pytest.mark.parametrize("experts,top_k,opts", [(200, 8, {}), (200, 8, dict(sigmoid=True)), (1024, 64, dict(sigmoid=True)),
                                                (256, 64, {}), (256, 8, dict(sigmoid=True, n_group=8, topk_group=4, group_top=2))])
def test_all_scores_close_together(experts, top_k, opts):
    """More scores within a binary32 rounding of each other than a wave has lanes, some of them equal in binary64 too."""
    dev = device()
    import torch
    say("route all close", experts, top_k, opts)
    rng = np.random.default_rng(experts + top_k)
    l = (np.float32(0.5) + np.float32(6e-8) * rng.integers(-8, 9, size=(20, experts))).astype(np.float32)
    l[1] = 0.5
    l[2, ::7] = -np.inf
    bias = (np.float32(0.01) + np.float32(1e-9) * rng.integers(0, 3, size=experts)).astype(np.float32)
    _check(torch, dev, l, top_k, dict(opts, bias=bias))
    _check(torch, dev, l, top_k, dict(opts, bias=np.zeros(experts, np.float32)))


@pytest.mark.parametrize("tokens,experts,top_k", [(1, 1, 1), (1, 128, 8), (64, 128, 8), (7, 3, 3), (1000, 60, 5), (4099, 257, 7),
                                                  (16384, 256, 8), (3, 1024, 64), (20000, 33, 8), (33000, 7, 4)])
def test_group_matches_oracle(tokens, experts, top_k):
    dev = device()
    import torch
    say("group", tokens, experts, top_k)
    rng = np.random.default_rng(tokens + experts)
    sel = rng.integers(-1, experts + 1, size=(tokens, top_k)).astype(np.int32)     # some ids are no expert
    sel[rng.random(sel.shape) < 0.02] = -(1 << 31)
    offsets = torch.full((experts + 3,), 77, dtype=torch.int32, device=dev)
    order = torch.full((sel.size + 2,), 77, dtype=torch.int32, device=dev)
    tg.moe_group(torch.from_numpy(sel).to(dev), experts, offsets=offsets[1:-1], order=order[1:-1])
    torch.cuda.synchronize()
    off, ordr = oracle.group(sel, experts)
    o, r = offsets.cpu().numpy(), order.cpu().numpy()
    assert np.array_equal(o[1:-1], off) and np.array_equal(r[1:-1], ordr)
    assert o[0] == o[-1] == r[0] == r[-1] == 77


@pytest.mark.parametrize("pairs,experts,taken", [(1 << 17, 256, 255), (1 << 17, 256, 0), (1 << 17, 512, -1), (1 << 17, 3, 2),
                                                 ((1 << 17) + 1, 256, 17), ((1 << 17) - 1, 256, -1), (700001, 256, 255), (700001, 40, 40)])
def test_long_runs_of_one_id(pairs, experts, taken):
    """Whole stretches of one id (an expert's, or none's) between random ones: every bit of a lane's batch is a hit."""
    dev = device()
    import torch
    say("group runs", pairs, experts, taken)
    rng = np.random.default_rng(pairs + experts)
    sel = rng.integers(0, experts, size=(pairs, 1)).astype(np.int32)
    sel[1000:pairs // 2] = taken
    sel[pairs // 2 + 77:pairs - 5] = taken
    for shift in (0, 1):                                             # aligned ids, and ids read one by one
        t = torch.empty(pairs + shift, dtype=torch.int32, device=dev)[shift:]
        t.copy_(torch.from_numpy(sel[:, 0]))
        offsets, order = tg.moe_group(t, experts)
        off, ordr = oracle.group(sel, experts)
        assert np.array_equal(offsets.cpu().numpy(), off) and np.array_equal(order.cpu().numpy(), ordr)


def test_one_expert_takes_all():
    dev = device()
    import torch
    say("group one expert")
    for e in (0, 6):
        off, order = tg.moe_group(torch.full((300, 2), e, dtype=torch.int32, device=dev), 7)
        assert order.tolist() == list(range(600))
        assert off.tolist() == [0] * (e + 1) + [600] * (7 - e)
