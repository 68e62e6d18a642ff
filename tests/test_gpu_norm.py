"""rms_norm on the GPU against the oracle: the sum and the steps exact, scales and outputs within their roundings."""
import numpy as np
import pytest

from gpu_common import device, say
from oracle import fp8, norm
from trellis_coded_gemv_amd import binding as tg

pytestmark = pytest.mark.gpu

# A step is 2^-24, the rounding of a binary32. Eight squares are summed in binary32, each rounded and added with one rounding (a fused
# multiply-add), all of one sign: 8 steps of their sum at most, and so of the mean, 4 of r, its root's reciprocal (the rest of the mean
# is binary64's). A scale is rounded once behind that: 5 steps. An output is rounded with r and with two products: 7 steps; a 16-bit one once more by half a
# step of its type, below the normal range by half of the smallest one. SLACK: second-order terms and binary64's roundings.
STEP = 2.0 ** -24
HALF = {"float32": (0.0, 2.0 ** -149), "float16": (2.0 ** -11, 2.0 ** -25), "bfloat16": (2.0 ** -8, 2.0 ** -133)}
SLACK = 2.0 ** -36


def _rows(torch, rows, n, pad, dtype, dev, seed, scale=1.0):
    x = torch.randn(rows, n + pad, generator=torch.Generator().manual_seed(seed)) * scale
    x[:, :: 97] *= 12
    x = x.to(getattr(torch, dtype))
    if pad:
        x[:, n:] = float("nan")                                     # between the rows: never read
    return x.to(dev)[:, :n]


def _wide(torch, rows, n, pad, dtype, dev):
    """An output of rows in a larger buffer whose rest must stay as it is."""
    buf = torch.full((rows + 2, n + pad), 99, device=dev).to(dtype)
    return buf, buf[1:-1, :n]


def _untouched(buf, n):
    b = buf.double()
    return bool((b[0] == b[0, 0]).all() and (b[-1] == b[0, 0]).all() and (b[:, n:] == b[0, 0]).all())


def _check(torch, x, w, residual, eps, out, y, scales, total):
    """Against the oracle, on a choice of rows."""
    rows = x.shape[0]
    pick = np.arange(rows) if rows <= 8 else np.unique(np.r_[0, 1, rows // 2, rows - 2, rows - 1])
    host = lambda t: t[torch.from_numpy(pick).to(t.device)].double().cpu().numpy()
    kind = None if residual is None else str(residual.dtype).split(".")[1]
    h, r, v = norm.rms_norm(host(x), w.double().cpu().numpy(), None if residual is None else host(residual), eps, kind)
    if residual is not None:
        assert np.array_equal(host(total), h, equal_nan=True)
    bad = np.isnan(r)
    if out == "int8":
        q, amax = norm.steps127(np.where(bad[:, None], 0.0, v))
        assert np.array_equal(host(y), q)
        want = np.where(bad, np.nan, amax * r / 127)
    elif out == "float8_e4m3fn":
        codes, s = fp8.quantize(np.where(bad[:, None], 0.0, v))
        assert np.array_equal(y.view(torch.uint8)[torch.from_numpy(pick).to(y.device)].cpu().numpy() & 0x7F, codes & 0x7F)
        assert np.array_equal(host(y.float()), fp8.values(codes))
        want = np.where(bad[:, None], np.nan, s * r[:, None])
    else:
        got, want = host(y), np.where(bad[:, None], np.nan, v * r[:, None])
        assert np.array_equal(np.isnan(got), np.isnan(want))
        rel, least = HALF[out]
        assert np.all((np.abs(got - want) <= np.abs(want) * ((1 + 7 * STEP) * (1 + rel) - 1 + SLACK) + least + 2.0 ** -149)[~np.isnan(want)])
        return
    got = host(scales)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.all((np.abs(got - want) <= np.abs(want) * (5 * STEP + SLACK) + 2.0 ** -149)[~np.isnan(want)])


OUTS = ["float32", "float16", "bfloat16", "int8", "float8_e4m3fn"]


@pytest.mark.parametrize("rows,n,pad", [(1, 1, 0), (3, 7, 1), (1, 16, 0), (5, 127, 0), (4, 128, 8), (2, 129, 3), (3, 512, 0), (2, 513, 2), (7, 1024, 0),
                                        (2, 1025, 1), (1, 2048, 0), (3, 2056, 0), (2, 4097, 5), (1, 8192, 0), (2, 8200, 0), (3, 16384, 0), (2, 16385, 1),
                                        (1, 32768, 0), (2, 32767, 3), (600, 4096, 0), (513, 5001, 1), (515, 8192, 0), (520, 10240, 0),
                                        (514, 10247, 3), (512, 12288, 0), (513, 16383, 1), (3, 24576, 0), (2, 20001, 0), (66000, 40, 0)])
@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_rows(rows, n, pad, out, dtype):
    dev = device()
    import torch
    say("norm", rows, n, pad, out, dtype)
    other = {"float32": "bfloat16", "float16": "float32", "bfloat16": "bfloat16"}[dtype]
    x, res = _rows(torch, rows, n, pad, dtype, dev, n), _rows(torch, rows, n, pad + 1, other, dev, n + 1, 3.0)
    w = (torch.rand(n, generator=torch.Generator().manual_seed(n)) + 0.5).to(getattr(torch, dtype if n % 2 else "float32")).to(dev)
    odt = getattr(torch, out)
    ybuf, y = _wide(torch, rows, n, pad + 3, odt, dev)
    tbuf, total = _wide(torch, rows, n, pad + 2, getattr(torch, other), dev)
    kw = dict(y=y, total=total)
    if out == "int8":
        kw["scales"] = torch.full((rows,), 99.0, device=dev)
    elif out == "float8_e4m3fn":
        sbuf, kw["scales"] = _wide(torch, rows, -(-n // 128), 2, torch.float32, dev)
    got = tg.rms_norm(x, w, residual=res, eps=1e-5, out_dtype=odt, **kw)
    torch.cuda.synchronize()
    assert got[-1] is total and got[0] is y
    _check(torch, x, w, res, float(np.float32(1e-5)), out, y, kw.get("scales"), total)
    assert _untouched(ybuf, n) and _untouched(tbuf, n) and (out != "float8_e4m3fn" or _untouched(sbuf, -(-n // 128)))
    alone = tg.rms_norm(x, w, out_dtype=odt)                        # without a residual
    torch.cuda.synchronize()
    y, scales = alone if isinstance(alone, tuple) else (alone, None)
    _check(torch, x, w, None, float(np.float32(1e-6)), out, y, scales, None)


@pytest.mark.parametrize("residual", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("weight", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_types(dtype, residual, weight):
    dev = device()
    import torch
    say("norm types", dtype, residual, weight)
    x, res = _rows(torch, 3, 1003, 0, dtype, dev, 1), _rows(torch, 3, 1003, 0, residual, dev, 2)
    w = torch.randn(1003, generator=torch.Generator().manual_seed(3)).to(getattr(torch, weight)).to(dev)
    for out in OUTS:
        got = tg.rms_norm(x, w, residual=res, out_dtype=getattr(torch, out))
        _check(torch, x, w, res, float(np.float32(1e-6)), out, got[0], got[1] if len(got) == 3 else None, got[-1])


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("n", [40, 300, 9000])
def test_special_rows(n, dtype, out):
    """Zeros, NaN, infinities, one value, the type's largest and smallest values, sums that leave the type; eps 0."""
    dev = device()
    import torch
    say("norm special", n, dtype, out)
    t = getattr(torch, dtype)
    fi = torch.finfo(t)
    g = torch.Generator().manual_seed(1)
    x, res = torch.randn(10, n, generator=g).to(t), torch.zeros(10, n, dtype=t)
    x[0] = 0
    x[1, n - 1] = float("nan")
    x[2, 5] = float("-inf")
    x[3] = 0
    x[3, n - 2] = -2.5
    x[4, 3] = fi.max
    x[5] = 0
    x[5, :4] = torch.tensor([fi.smallest_normal, -fi.smallest_normal / 2, fi.smallest_normal / 4, 0]).to(t)
    x[6] = -0.0
    x[7] = fi.max
    x[8] *= fi.tiny
    x[9, 0] = res[9, 0] = fi.max                                    # the sum is an infinity
    w = (torch.rand(n, generator=g) + 0.5).to(t)
    x, res, w = x.to(dev), res.to(dev), w.to(dev)
    for eps in (0.0, 1e-6):
        got = tg.rms_norm(x, w, residual=res, eps=eps, out_dtype=getattr(torch, out))
        torch.cuda.synchronize()
        _check_special(torch, x, w, res, eps, out, got)


def _check_special(torch, x, w, res, eps, out, got):
    # more than 48 significant bits are possible nowhere; rows of values near the type's ends go through the same check
    _check(torch, x[:8], w, res[:8], float(np.float32(eps)), out, got[0][:8], got[1][:8] if len(got) == 3 else None, got[-1][:8])
    _check(torch, x[8:], w, res[8:], float(np.float32(eps)), out, got[0][8:], got[1][8:] if len(got) == 3 else None, got[-1][8:])


@pytest.mark.parametrize("out", OUTS)
def test_weights_that_are_not_finite(out):
    """They reach their own value, the scale of their own 128 values, or that of the row (int8)."""
    dev = device()
    import torch
    say("norm weights", out)
    x = torch.randn(4, 400, generator=torch.Generator().manual_seed(5)).half().to(dev)
    w = torch.ones(400, device=dev)
    w[130] = float("nan")
    w[131] = float("inf")
    got = tg.rms_norm(x, w, out_dtype=getattr(torch, out))
    clean = tg.rms_norm(x, torch.ones(400, device=dev), out_dtype=getattr(torch, out))
    torch.cuda.synchronize()
    if out == "int8":
        assert got[1].isnan().all() and not got[0].any()
    elif out == "float8_e4m3fn":
        assert got[1][:, 1].isnan().all() and torch.equal(got[1][:, [0, 2, 3]], clean[1][:, [0, 2, 3]])
        q, c = got[0].float(), clean[0].float()
        assert not q[:, 128:256].any() and torch.equal(q[:, :128], c[:, :128]) and torch.equal(q[:, 256:], c[:, 256:])
    else:
        assert got[:, 130].isnan().all() and got[:, 131].isinf().all()
        assert torch.equal(got[:, :130], clean[:, :130]) and torch.equal(got[:, 132:], clean[:, 132:])


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("out", ["int8", "float8_e4m3fn"])
def test_steps_on_the_borders(out, dtype):
    """Products that lie on the borders of two steps, and next to them by a last place."""
    dev = device()
    import torch
    say("norm borders", out, dtype)
    t = getattr(torch, dtype)
    m = fp8.magnitudes()
    top, mid = (127.0, np.arange(0.5, 127)) if out == "int8" else (448.0, (m[1:] + m[:-1]) / 2)
    n = len(mid) + 2
    rows = []
    for scale in (1.0, 2.0 ** -5, 3.0):                             # 3: the row's largest is no power of two times the step
        v = torch.from_numpy(np.r_[top, mid, -mid[3]] * scale).to(t)
        rows += [v, -v, v * (1 + 2 * torch.finfo(t).eps), v * (1 - torch.finfo(t).eps)]
        rows[-1][0] = rows[-2][0] = v[0]
    x = torch.stack(rows).to(t)
    pieces = [x[:, :1].expand(-1, 128).clone() for _ in range(-(-n // 126))]    # each 128 values with the largest among them
    for i, p in enumerate(pieces):
        part = x[:, 126 * i:126 * i + 126]
        p[:, 2:2 + part.shape[1]] = part
    x = torch.cat(pieces, 1).contiguous().to(dev)
    for w in (torch.ones(x.shape[1]), torch.full((x.shape[1],), 1.0 + 2.0 ** -7)):
        w = w.to(t).to(dev)
        got = tg.rms_norm(x, w, out_dtype=getattr(torch, out))
        torch.cuda.synchronize()
        _check(torch, x, w, None, float(np.float32(1e-6)), out, got[0], got[1], None)
        for r in range(8, x.shape[0]):
            _check(torch, x[r:r + 1], w, None, float(np.float32(1e-6)), out, got[0][r:r + 1], got[1][r:r + 1], None)


def test_in_place_and_shapes():
    dev = device()
    import torch
    say("norm in place")
    g = torch.Generator().manual_seed(9)
    x, res = torch.randn(2, 3, 200, generator=g).to(dev), torch.randn(2, 3, 200, generator=g).bfloat16().to(dev)
    w = torch.rand(200, generator=g).to(dev)
    y, total = tg.rms_norm(x, w, residual=res)
    assert y.shape == total.shape == x.shape and y.dtype == torch.float32 and total.dtype == torch.bfloat16
    q, s, t2 = tg.rms_norm(x, w, residual=res, out_dtype=torch.float8_e4m3fn)
    assert q.shape == x.shape and s.shape == (2, 3, 2) and torch.equal(t2, total)
    q8, s8, _ = tg.rms_norm(x, w, residual=res, out_dtype=torch.int8)
    assert q8.shape == x.shape and s8.shape == (2, 3)
    stream = res.clone()
    y2, t3 = tg.rms_norm(x, w, residual=stream, total=stream)
    assert t3 is stream and torch.equal(stream, total) and torch.equal(y2, y)
    xs = x.bfloat16()
    y3, _ = tg.rms_norm(xs, w, residual=res)
    sum_in_x = xs.clone()
    y4, _ = tg.rms_norm(sum_in_x, w, residual=res, total=sum_in_x)
    assert torch.equal(y4, y3) and torch.equal(sum_in_x, (xs.float() + res.float()).bfloat16())
    one = tg.rms_norm(x[1, 2], w)
    assert one.shape == (200,) and torch.equal(one, tg.rms_norm(x, w)[1, 2])
    assert torch.equal(tg.rms_norm(x.transpose(0, 1), w), tg.rms_norm(x, w).transpose(0, 1))
    cols = x[:, :, 0].t()                                           # the innermost stride is not one
    assert torch.equal(tg.rms_norm(cols, w[:2]), tg.rms_norm(cols.contiguous(), w[:2]))
    with pytest.raises(tg.TgError):
        tg.rms_norm(x[0, :1].expand(4, 200), w)                     # rows that share their memory
