"""moe_route_scored at the ends of the range: weights whose scores lie below fp32's, against a
plain 64-bit reference, compared relatively."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from sparse_moe_layer_row_gb300 import moe_block as mb
from tests import fp8_ref as F

pytestmark = pytest.mark.gpu

U = 2.0 ** -24   # half a step of fp32
# A renormalised weight: the exponential (2 ulp = 4 U), the low part of its argument (1), 1 + e^z
# (its exponential's 4 at most, and 1) and that quotient (1): 11; the sum of such numbers, five
# additions deep: 16; the quotient and the scale: 2.  A weight below 2^-126: a step 2^-149 more for
# each of its last two roundings.
RTOL_W = 29 * U
ATOL_W = 2 * 2.0 ** -149
# A sigmoid: its exponential 4 U, 1 + e^-z and the quotient 1 each; below 2^-126 two of the least
# steps of the exponential and half a one.  Under the softmax the argument z - m is rounded
# (|z - m| U), and e^(z - m) is multiplied by one over the sum (the sum of fast exponentials:
# 3e-6 as in the other tests of this call).
ATOL_S = 3 * 2.0 ** -149


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    mb.load()


def run(z, rule, k, bias=None):
    R = z.shape[0]
    idx = torch.full((R, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((R, k), float("nan"), device="cuda")
    s = torch.full((R, k), float("nan"), device="cuda")
    mb.moe_route_scored(z, rule, idx, w, select_bias=bias, topk_score=s)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().double().numpy(), s.cpu().double().numpy()


def check(z, rule, k, bias=None):
    idx, w, s = run(z, rule, k, bias)
    zn = z.double().cpu().numpy()
    bn = None if bias is None else bias.double().cpu().numpy()
    for r in range(z.shape[0]):
        ri, rw, rs = F.route(zn[r], rule, k, bn)
        assert np.array_equal(idx[r], ri), (r, idx[r], ri)
        ts, far = 6 * U, zn[r][ri][rs > 0]
        if rule.score == "softmax" and len(far):
            ts = 3e-6 + U * float(np.max(zn[r]) - far.min())
        assert np.all(np.abs(s[r] - rs) <= ts * rs + ATOL_S), (r, s[r], rs)
        if rule.renormalize:
            assert np.all(np.abs(w[r] - rw) <= RTOL_W * rw + ATOL_W * rule.scale), (r, w[r], rw)
        else:
            assert np.all(np.abs(w[r] - rw) <= (ts + U) * rw + (ATOL_S + 2.0 ** -149) * rule.scale), (r, w[r], rw)


def uniform(R, E, lo, hi, seed=0, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (lo + (hi - lo) * torch.rand(R, E, generator=g, device="cuda")).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("lo,hi", [(-85.0, -70.0), (-100.0, -80.0), (-300.0, -85.0), (-690.0, -680.0)])
@pytest.mark.parametrize("scale", [1.0, 2.5])
def test_sigmoid_rows_of_very_low_logits(lo, hi, scale, dtype):
    """Every score of the row is near or below the least fp32 number: the weights are their
    ratios all the same."""
    z = uniform(40, 64, lo, hi, seed=int(-lo), dtype=dtype)
    check(z, mb.RouteRule(score="sigmoid", scale=scale), 8)
    check(z, mb.RouteRule(score="sigmoid", scale=scale), 1)
    check(z, mb.RouteRule(score="sigmoid", scale=scale, renormalize=False), 8)


def test_sigmoid_equal_low_logits_share_evenly():
    z = torch.full((3, 64), -95.0, device="cuda")
    z[1] = -100.0
    z[1, 5] = -101.0
    z[2, 8:] = float("-inf")
    idx, w, _ = run(z, mb.RouteRule(score="sigmoid"), 8)
    assert np.all(w[0] == 0.125) and np.all(w[1] == 0.125) and np.all(w[2] == 0.125)
    two = torch.full((1, 16), float("-inf"), device="cuda")
    two[0, 3], two[0, 9] = -100.0, -101.0
    idx, w, _ = run(two, mb.RouteRule(score="sigmoid"), 4)
    assert list(idx[0]) == [3, 9, 0, 1] and not w[0, 2:].any()
    ref = np.array([1.0, np.exp(-1.0)]) / (1.0 + np.exp(-1.0))
    assert np.all(np.abs(w[0, :2] - ref) <= RTOL_W * ref)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_bias_picks_experts_far_below(score, renormalize):
    """The bias takes experts whose scores are 1e-33 .. 1e-65, of the row's largest, which is not
    taken, under the softmax; some rows take one of ordinary size beside them."""
    R, E, k = 48, 64, 8
    z = uniform(R, E, -150.0, -90.0, seed=3)
    z[:, 32:] = uniform(R, 32, -1.0, 3.0, seed=4)
    if score == "sigmoid":
        z[:, 32:] -= 50.0
    z[::4, 9] = uniform(12, 1, -2.0, 2.0, seed=5)[:, 0]
    z[1::4, 30] = float("-inf")
    z[2::4, 24:32] = -75.0 - torch.arange(8, device="cuda") * 2.0
    bias = torch.full((E,), -4.0, device="cuda")
    bias[:32] = 1.0 + torch.arange(32, device="cuda") * 2.0 ** -4   # scores do not reach these steps
    bias[9] = 9.0
    check(z, mb.RouteRule(score=score, renormalize=renormalize, scale=2.0), k, bias)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_scores_that_are_zero_in_64_bits_weigh_nothing(score):
    """Logits of the type's lowest value are masks in effect: chosen, they have weight 0; a row
    with nothing else has weights 0 (sigmoid) or, under the softmax, shares evenly."""
    low = torch.finfo(torch.float32).min
    z = torch.full((3, 32), low, device="cuda")
    z[1, 3] = -95.0
    z[2, 3], z[2, 4] = 1.0, float("-inf")
    check(z, mb.RouteRule(score=score), 4)
    bias = torch.linspace(0.0, 1.0, 32, device="cuda")
    check(z, mb.RouteRule(score=score), 4, bias)


def test_ordinary_rows_keep_ratios_across_the_border():
    """Chosen scores on both sides of where the ratio form takes over."""
    z = uniform(200, 32, -72.0, -66.0, seed=11)
    z[::3, :4] = uniform(67, 4, -3.0, 3.0, seed=12)
    check(z, mb.RouteRule(score="sigmoid"), 8)
