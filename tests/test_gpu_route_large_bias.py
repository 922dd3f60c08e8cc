"""moe_route_scored with selection biases near the largest finite fp32 values: sums of two keys
pass fp32's range, and the order is still that of the real values."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from sparse_moe_layer_row_gb300 import moe_block as mb
from tests import fp8_ref as F

pytestmark = pytest.mark.gpu
BIG = torch.finfo(torch.float32).max
# a weight: 3e-6 as in the other tests of this call, and half a step of an argument z - m within 16
RTOL = 3e-6 + 16 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    mb.load()


def biases(kind, E, G):
    g = torch.Generator(device="cuda").manual_seed(E + G)
    u = torch.rand(E, generator=g, device="cuda")
    if kind == "all largest":
        return torch.full((E,), BIG, device="cuda")
    if kind == "all lowest":
        return torch.full((E,), -BIG, device="cuda")
    if kind == "sums above":                     # every group's sum is above BIG, all apart
        return 2e38 + 1.3e38 * u
    if kind == "sums below":
        return -2e38 - 1.3e38 * u
    if kind == "around the border":
        return (1.4e38 + 0.6e38 * u)
    b = (u - 0.5) * 0.1                          # ordinary, but for two forced and two barred groups
    n = E // G
    b[n:2 * n] = BIG
    b[3 * n:4 * n] = BIG
    b[:n] = -BIG
    b[-n:] = -BIG
    return b


@pytest.mark.parametrize("kind", ["all largest", "all lowest", "sums above", "sums below", "around the border",
                                  "forced and barred"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,top", [(64, 8, 3), (256, 8, 4), (48, 6, 5), (1024, 32, 31)])
def test_order_of_large_sums(E, G, top, score, kind):
    R, k = 24, 8
    g = torch.Generator(device="cuda").manual_seed(5)
    z = torch.randn(R, E, generator=g, device="cuda")
    z[R // 2, : 2 * (E // G)] = float("-inf")    # groups that are masked throughout
    z[R // 2 + 1, ::2] = float("-inf")
    bias = biases(kind, E, G)
    zn, bn = z.double().cpu().numpy(), bias.double().cpu().numpy()
    for gscore in ("top2", "max"):
        rule = mb.RouteRule(score=score, n_groups=G, top_groups=top, group_score=gscore)
        idx = torch.full((R, k), -7, dtype=torch.int32, device="cuda")
        w = torch.full((R, k), float("nan"), device="cuda")
        mb.moe_route_scored(z, rule, idx, w, select_bias=bias)
        torch.cuda.synchronize()
        got, gw = idx.cpu().numpy(), w.cpu().double().numpy()
        for r in range(R):
            ri, rw, _ = F.route(zn[r], rule, k, bn)
            assert np.array_equal(got[r], ri), (gscore, r, got[r], ri)
            assert np.all(np.abs(gw[r] - rw) <= RTOL * np.abs(rw)), (gscore, r)
