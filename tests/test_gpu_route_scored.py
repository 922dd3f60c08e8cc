"""moe_route_scored against a plain 64-bit reference: scores, bias, groups, masks, ties,
types and strides; and moe_block_logits with it on a plan."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from sparse_moe_layer_row_gb300 import moe_block as mb, workloads as W
from tests import fp8_ref as F

pytestmark = pytest.mark.gpu

# A weight is a quotient of scores: the score's exponential (2 ulp), its sum and quotient,
# the sum of at most 32 scores, the quotient and the scale.  The softmax's sum of E fast
# exponentials: each 2^-22 + |z - m| 2^-23 of itself, at most 1e-6 of the sum (the far ones
# weigh nothing); together under 3e-6 of the weight.  A softmax numerator e^{z - m} also has the
# rounding of z - m, half a step of it: the check adds 2^-24 |z - m| of the farthest one chosen.
RTOL = 3e-6


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    mb.load()


def run(z, rule, k, bias=None, scores=True):
    R = z.shape[0]
    idx = torch.full((R, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((R, k), float("nan"), device="cuda")
    s = torch.full((R, k), float("nan"), device="cuda") if scores else None
    mb.moe_route_scored(z, rule, idx, w, select_bias=bias, topk_score=s)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().double().numpy(), s.cpu().double().numpy() if scores else None


def check(z, rule, k, bias=None):
    idx, w, s = run(z, rule, k, bias)
    zn = z.double().cpu().numpy()
    bn = None if bias is None else bias.double().cpu().numpy()
    for r in range(z.shape[0]):
        ri, rw, rs = F.route(zn[r], rule, k, bn)
        assert np.array_equal(idx[r], ri), (r, idx[r], ri)
        t = RTOL
        far = zn[r][ri][rs > 0]
        if rule.score == "softmax" and len(far) and np.isfinite(zn[r]).any() and not np.isinf(far).any():
            t += 2.0 ** -24 * float(np.nanmax(zn[r]) - far.min())
        assert np.all(np.abs(w[r] - rw) <= t * np.abs(rw) + 1e-37), (r, w[r], rw)
        assert np.all(np.abs(s[r] - rs) <= t * np.abs(rs) + 1e-37), (r, s[r], rs)


def logits(R, E, dtype=torch.float32, seed=0, sigma=0.9):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(R, E, generator=g, device="cuda") * sigma).to(dtype)


def bias_of(E, seed=1, sigma=0.05):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(E, generator=g, device="cuda") * sigma


RULES = [
    mb.RouteRule(),
    mb.RouteRule(score="softmax", renormalize=False),
    mb.RouteRule(score="sigmoid", scale=2.5),
    mb.RouteRule(score="sigmoid", n_groups=8, top_groups=4, group_score="top2", scale=2.5),
    mb.RouteRule(score="softmax", n_groups=8, top_groups=3, group_score="max", renormalize=False, scale=16.0),
    mb.RouteRule(score="softmax", n_groups=4, top_groups=1, group_score="top2"),
    mb.RouteRule(score="sigmoid", n_groups=2, top_groups=2, group_score="max"),
]


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("rule", RULES, ids=lambda r: f"{r.score}-g{r.n_groups}t{r.top_groups}{r.group_score}")
@pytest.mark.parametrize("R,E,k,dtype", [(1, 256, 8, torch.float32), (33, 256, 8, torch.bfloat16),
                                         (300, 160, 6, torch.float32), (5, 32, 2, torch.float16),
                                         (3, 1024, 32, torch.float32), (40, 24, 3, torch.bfloat16),
                                         (7, 512, 16, torch.float16)])
def test_matches_reference(R, E, k, dtype, rule, biased):
    if k > rule.top_groups * (E // rule.n_groups):
        pytest.skip("more experts than the groups hold")
    check(logits(R, E, dtype, seed=R + E), rule, k, bias_of(E) if biased else None)


@pytest.mark.parametrize("rule", RULES, ids=lambda r: f"{r.score}-g{r.n_groups}t{r.top_groups}{r.group_score}")
def test_many_rows(rule):
    """Enough rows that some have neighbours too close for 32 bits."""
    z, b = logits(4000, 256, seed=9), bias_of(256)
    check(z, rule, 8, b)
    check(z, rule, 8)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_near_ties_order_by_real_value(score):
    """Keys a few units of 2^-30 apart: equal in 32 bits, ordered in 64.  The bias pulls
    unlike scores to almost the same key."""
    E = 64
    z = logits(64, E, seed=4)
    zd = z.double()
    s = torch.sigmoid(zd) if score == "sigmoid" else torch.softmax(zd, 1)
    bias = (0.75 - s[0]).float()   # row 0: every key near 0.75, apart by the bias's roundings
    check(z, mb.RouteRule(score=score), 8, bias)
    check(z, mb.RouteRule(score=score, n_groups=8, top_groups=3, group_score="top2"), 8, bias)
    check(z, mb.RouteRule(score=score, n_groups=8, top_groups=3, group_score="max"), 8, bias)


@pytest.mark.parametrize("rule", RULES, ids=lambda r: f"{r.score}-g{r.n_groups}t{r.top_groups}{r.group_score}")
@pytest.mark.parametrize("biased", [False, True])
def test_ties_masks_and_specials(rule, biased):
    """Equal logits, masked experts, rows masked but for one expert or throughout, NaN,
    +inf, zeros of both signs, very large logits."""
    E, k = 64, 8
    z = logits(16, E, seed=2)
    z[0] = 0.5                                   # all equal: the lowest ids
    z[1] = float("-inf")                         # nothing left
    z[2] = float("-inf")
    z[2, 37] = 1.0                               # one expert left
    z[3, ::2] = float("-inf")
    z[4, 5] = float("nan")
    z[5] = float("nan")
    z[6, :20] = float("-inf")
    z[6, 40:] = float("nan")
    z[7, 11] = float("inf")
    z[8] = 0.0
    z[8, ::3] = -0.0
    z[9] = torch.round(z[9])                     # many ties
    z[10] *= 30.0
    z[11] = -40.0 + torch.arange(E, device="cuda") * 0.25
    z[12] = torch.finfo(torch.float32).min       # the type's lowest value is no mask
    z[13, 3] = float("inf")
    z[13, 50] = float("inf")
    if rule.score == "sigmoid":
        z[10] = z[10].clamp(-20, 20)             # beyond, 64-bit sigmoids of unlike logits are equal too
    bias = bias_of(E, sigma=0.3) if biased else None
    check(z, rule, k, bias)


def test_zero_bias_is_no_bias_on_ties():
    z = torch.round(logits(50, 128, seed=6) * 4) / 4
    zero = torch.zeros(128, device="cuda")
    for rule in RULES:
        a, b = run(z, rule, 8, zero), run(z, rule, 8)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_strided_rows_streams_and_repeats():
    wide = logits(70, 300, seed=3)
    z = wide[:, 20:276]
    rule, b = RULES[3], bias_of(256)
    a = run(z, rule, 8, b)
    c = run(z.contiguous(), rule, 8, b, scores=False)
    assert np.array_equal(a[0], c[0]) and np.array_equal(a[1], c[1])
    st = torch.cuda.Stream()
    idx = torch.empty(70, 8, dtype=torch.int32, device="cuda")
    w = torch.empty(70, 8, device="cuda")
    st.wait_stream(torch.cuda.current_stream())
    mb.moe_route_scored(z, rule, idx, w, select_bias=b, stream=st)
    st.synchronize()
    assert np.array_equal(idx.cpu().numpy(), a[0]) and np.array_equal(w.cpu().double().numpy(), a[1])
    odd = logits(9, 33, torch.bfloat16, seed=8)[:, :31]   # rows on odd 2-byte offsets
    check(odd, mb.RouteRule(score="sigmoid"), 4)


def test_no_rows():
    z = torch.empty(0, 64, device="cuda")
    assert run(z, RULES[0], 4)[0].shape == (0, 4)


def test_graph_capture():
    z, rule, b = logits(32, 256, seed=5), RULES[3], bias_of(256)
    idx = torch.empty(32, 8, dtype=torch.int32, device="cuda")
    w = torch.empty(32, 8, device="cuda")
    mb.moe_route_scored(z, rule, idx, w, select_bias=b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mb.moe_route_scored(z, rule, idx, w, select_bias=b)
    z.copy_(logits(32, 256, seed=50))
    g.replay()
    torch.cuda.synchronize()
    ref = run(z, rule, 8, b)
    assert np.array_equal(idx.cpu().numpy(), ref[0]) and np.array_equal(w.cpu().double().numpy(), ref[1])


def layer_of(w):
    T = W.make_tensors(w, device="cuda")
    return T, mb.MoeBlockLayer(T.w_router, T.w_gate, T.w_up, T.w_down, T.ws_gate, T.ws_up, T.ws_down,
                               k=w.k, max_rows=w.R, max_blocks=w.nb)


@pytest.mark.parametrize("w", [W.TINY, W.BLOCKS16_ZIPF, W.BY_NAME["rows2048-b32-tau0.9"]], ids=lambda w: w.name)
def test_block_logits(w):
    """The logits against 64 bits.  H products, exact in fp32, are added in fp32: each addition
    a whole step 2^-23 of the sum of magnitudes at most (a tensor core may truncate), and the
    bias half a step."""
    T, layer = layer_of(w)
    z = torch.full((w.R, w.E), float("nan"), device="cuda")
    mb.moe_block_logits(layer.plan, T.x, T.block_offsets, T.bias, z, layer.workspace)
    torch.cuda.synchronize()
    x, wr = T.x.double(), T.w_router.double()
    ref, mag = x @ wr.t(), x.abs() @ wr.abs().t()
    if T.bias is not None:
        block = torch.searchsorted(T.block_offsets, torch.arange(w.R, device="cuda"), right=True) - 1
        ref = ref + T.bias.double()[block]
    assert torch.all((z.double() - ref).abs() <= w.H * F.STEP * mag + ref.abs() * 2.0 ** -24)
    assert layer.status()["nonfinite_logits"] == 0
    T.x[3, 7] = float("nan")
    mb.moe_block_logits(layer.plan, T.x, T.block_offsets, T.bias, z, layer.workspace)
    torch.cuda.synchronize()
    assert torch.isnan(z[3]).all() and torch.isfinite(z[:3]).all() and torch.isfinite(z[4:]).all()
    assert layer.status()["nonfinite_logits"] == w.E


@pytest.mark.parametrize("w", [W.TINY, W.BLOCK32], ids=lambda w: w.name)
def test_layer_route_scored(w):
    """A plan's logits of up to 255 rows order as moe_block_route does (fixed order), and
    routing by the softmax rule over the chosen gives its weights."""
    T, layer = layer_of(w)
    idx0, w0 = (t.clone() for t in layer.route(T.x, T.block_offsets, T.bias))
    idx, wt, sc = layer.route_scored(T.x, T.block_offsets, mb.RouteRule(), bias=T.bias)
    torch.cuda.synchronize()
    assert torch.equal(idx, idx0)
    assert torch.all((wt - w0).abs() <= 2 * RTOL * w0)
    assert torch.all(sc.sum(1) <= 1.0 + 1e-5) and torch.all(sc > 0)
