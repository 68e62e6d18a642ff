"""moe_route within groups where a group's value is not what its binary32 sum says: biases that cancel, and biases whose sums leave the type."""
import numpy as np
import pytest

from gpu_common import device, say
from oracle import route as oracle
from trellis_coded_gemv_amd import binding as tg

pytestmark = pytest.mark.gpu

W_TOL = 2.0 ** -24 * (1 + 1e-6)     # one rounding to binary32 of a weight formed in binary64


def _check(torch, dev, l, top_k, bias, **kw):
    sel, w = tg.moe_route(torch.from_numpy(l).to(dev), top_k, bias=torch.from_numpy(bias).to(dev), **kw)
    ids, ref = oracle.route(l, top_k, bias=bias, **kw)
    wrong = np.flatnonzero((sel.cpu().numpy() != ids).any(1))
    assert wrong.size == 0, (wrong.size, l[wrong[0]], sel[wrong[0]].tolist(), ids[wrong[0]])
    assert np.all(np.abs(w.cpu().numpy().astype(np.float64) - ref) <= W_TOL * np.abs(ref) + 2.0 ** -150)


@pytest.mark.parametrize("B", [1.0, 64.0, 128.0, 1000.0, 1e5, 1e8, 1e30])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_cancelling_biases(B, sigmoid):
    """The two largest of a group are near B and -B: each is rounded relative to B, their sum is of the scores' size."""
    dev = device()
    import torch
    say("route groups cancelling", B, sigmoid)
    rng = np.random.default_rng(int(B) % 1000 + sigmoid)
    l = rng.normal(size=(3000, 4)).astype(np.float32)
    l[0] = [-0.01944458, 0.84007615, -0.63065845, 1.7055503]
    opts = dict(sigmoid=sigmoid, n_group=2, topk_group=1, group_top=2)
    _check(torch, dev, l, 2, np.array([B, -B, 0, 0], np.float32), **opts)
    _check(torch, dev, l, 2, np.array([0, 0, -B, B], np.float32), **opts)


@pytest.mark.parametrize("B", [300.0, 1e6])
@pytest.mark.parametrize("experts,n_group", [(64, 8), (60, 6), (256, 16)])
def test_a_far_group_of_large_biases(B, experts, n_group):
    """Some of many groups hold a pair of large biases that cancel; without them the groups lie close together."""
    dev = device()
    import torch
    say("route groups far", B, experts, n_group)
    rng = np.random.default_rng(experts)
    size = experts // n_group
    l = (rng.normal(size=(400, experts)) * 0.05).astype(np.float32)
    bias = np.zeros(experts, np.float32)
    bias[[size, size + 1, 3 * size, 3 * size + 1]] = [B, -B, -B, B]
    if size > 2:
        bias[size + 2:2 * size] = bias[3 * size + 2:4 * size] = -2 * B      # so that -B is their second largest
    for topk_group in (1, 2, n_group - 1, n_group):
        _check(torch, dev, l, 2, bias, sigmoid=True, n_group=n_group, topk_group=topk_group, group_top=2)


LOW, INF = float(np.finfo(np.float32).min), float("inf")


@pytest.mark.parametrize("bias", [
    [-INF, -INF, -3.4e38, -3.4e38], [-3.4e38, -3.4e38, -INF, -INF], [-INF, -INF, LOW, LOW, -INF, -INF, LOW, LOW], [LOW, LOW, -3.3e38, LOW],
    [LOW, LOW, LOW, LOW], [LOW, -INF, LOW, LOW, -INF, LOW, 0.0, LOW], [3.4e38, 3.4e38, 3.3e38, 3.4e38], [3.2e38, 3.3e38, 3.3e38, 3.3e38],
    [-LOW, LOW, 0.0, 0.0], [-INF, -LOW, -LOW, LOW, LOW, LOW, -INF, -INF]])
@pytest.mark.parametrize("group_top", [1, 2])
def test_values_that_leave_binary32(bias, group_top):
    """Sums of two lowest (or largest) biases are infinite in binary32 and numbers in binary64; groups without experts beside them."""
    dev = device()
    import torch
    say("route groups lowest", bias, group_top)
    rng = np.random.default_rng(7)
    l = rng.normal(size=(40, len(bias))).astype(np.float32)
    for topk_group in range(1, len(bias) // 2 + 1):
        for sigmoid in (True, False):
            _check(torch, dev, l, 2, np.array(bias, np.float32), sigmoid=sigmoid, n_group=len(bias) // 2, topk_group=topk_group, group_top=group_top)
