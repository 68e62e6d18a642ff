"""8-bit experts' products of more workgroups than one launch dimension holds."""
import pytest

from gpu_common import device, say
from trellis_coded_gemv_amd import binding as tg

pytestmark = pytest.mark.gpu

TOL = (1 + 2.0 ** -24) ** 3 * (1 + 2.0 ** -8) - 1   # three roundings to binary32 and one to bf16


@pytest.mark.parametrize("experts,m", [(1024, 1 << 20), (256, (1 << 22) - 3)])
def test_one_pair_for_each_of_many_wide_experts(experts, m):
    """17 GB of weights, 2^30 outputs: tiles of few rows, one list of them for every expert. Sampled outputs of all experts, and sums
    of whole rows' bits against the same products taken one expert at a time."""
    dev = device()
    import torch
    n = 16
    say("int8 grouped wide", experts, m)
    g = torch.Generator(device=dev).manual_seed(experts)
    wq = torch.empty(experts, m, n, dtype=torch.int8, device=dev)
    for e in range(0, experts, 64):
        wq[e:e + 64] = torch.randint(-128, 128, (min(64, experts - e), m, n), generator=g, device=dev, dtype=torch.int8)
    ws = torch.rand(experts, m, generator=g, device=dev) + 0.5
    xq = torch.randint(-128, 128, (experts, n), generator=g, device=dev, dtype=torch.int8)
    xs = torch.rand(experts, generator=g, device=dev) + 0.5
    sel = torch.randperm(experts, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    sel[5] = -1
    off, order = tg.moe_group(sel.to(dev), experts)
    y = tg.int8_gemm_grouped(tg.Int8Experts(wq, ws), xq, xs, off, order, out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    assert not bool(y[5].any())
    at = torch.tensor([0, 1, 31, 32, 63, 64, m // 2, m - 65, m - 2, m - 1], device=dev)
    for p, e in enumerate(sel.tolist()):
        if e < 0:
            continue
        ref = (wq[e, at].double() * xq[p].double()).sum(1) * xs[p].double() * ws[e, at].double()
        assert bool(((y[p, at].double() - ref).abs() <= TOL * ref.abs()).all()), p
        if p % 64 == 1:
            one = tg.int8_gemm(tg.Int8Layer(wq[e], ws[e]), xq[p:p + 1], xs[p:p + 1], out_dtype=torch.bfloat16)
            assert torch.equal(one[0], y[p]), p
