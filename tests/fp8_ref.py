"""Plain 64-bit references of the scored routing and the e4m3 block-scaled operators, and
the error bounds their tests use.

Bounds.  u = 2^-24 is half a step of fp32.  A product of two e4m3 codes is exact; a tensor
core may truncate where it aligns addends, so each addition counts as a whole step 2^-23 of
the sum of magnitudes.  A block of 128 then carries 128 of them, the fp32 promotion
2 (scale product, fma) per block, so that a sum over K is off by at most
(128 + 2 blocks + 2) 2^-23 S with S the sum of the magnitudes of its addends.
"""
from __future__ import annotations

import math

import numpy as np
import torch

BLOCK = 128
STEP = 2.0 ** -23
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}

E4M3 = np.array([m / 8 * 2.0 ** -6 for m in range(8)] +
                [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)])[:127]


def e4m3_round(v: torch.Tensor) -> torch.Tensor:
    """Nearest e4m3 value, halves to the even code; NaN stays NaN (|v| <= 448)."""
    t = torch.tensor(E4M3, dtype=torch.float64, device=v.device)
    a = v.abs()
    nan = torch.isnan(a)
    a = torch.where(nan, 0.0, a).contiguous()
    hi = torch.searchsorted(t, a).clamp(1, 126)
    lo = hi - 1
    mid = (t[lo] + t[hi]) / 2
    r = torch.where((a > mid) | ((a == mid) & (hi % 2 == 0)), t[hi], t[lo])
    return torch.where(nan, float("nan"), torch.where(v < 0, -r, r))


def e4m3_midpoint_gap(v: torch.Tensor):
    """Distance of |v| to the nearest midpoint between two codes, and that pair's step."""
    t = torch.tensor(E4M3, dtype=torch.float64, device=v.device)
    mids = (t[1:] + t[:-1]) / 2
    a = v.abs().contiguous()
    i = torch.searchsorted(mids, a).clamp(0, len(mids) - 1)
    j = (i - 1).clamp_min(0)
    di, dj = (mids[i] - a).abs(), (mids[j] - a).abs()
    k = torch.where(di <= dj, i, j)
    return torch.minimum(di, dj), t[k + 1] - t[k]


def pad_blocks(x: torch.Tensor) -> torch.Tensor:
    """[..., K] -> [..., blocks, 128], zeros after the end."""
    kb = -(-x.shape[-1] // BLOCK)
    x = torch.nn.functional.pad(x, (0, kb * BLOCK - x.shape[-1]))
    return x.view(*x.shape[:-1], kb, BLOCK)


def quantize(x: torch.Tensor):
    """Rows in fp64 -> codes (as values) [R, K] and scales [blocks, R] (fp32 numbers)."""
    R, K = x.shape
    p = pad_blocks(x.double())
    a = p.abs().amax(-1).clamp_min(2.0 ** -100)
    q = e4m3_round(448.0 * p / a[..., None]).view(R, -1)[:, :K]
    return q, (a / 448.0).float().double().t()


def row_values(q, s):
    """Codes [R, K] and scales [blocks, R] -> values in fp64."""
    f = s.double().t().repeat_interleave(BLOCK, -1)[:, :q.shape[1]]
    return q.double() * f


def weight_values(q, s):
    N, K = q.shape[-2:]
    f = s.double().repeat_interleave(BLOCK, -2)[..., :N, :].repeat_interleave(BLOCK, -1)[..., :K]
    return q.double() * f


def block_codes(w: torch.Tensor):
    """Weights [..., N, K] -> e4m3 codes and fp32 scales per 128 x 128 block (any valid codes do)."""
    *lead, N, K = w.shape
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    p = torch.nn.functional.pad(w.double(), (0, kb * BLOCK - K, 0, nb * BLOCK - N))
    p = p.view(*lead, nb, BLOCK, kb, BLOCK)
    s = (p.abs().amax(dim=(-3, -1)).clamp_min(2.0 ** -100) / 448.0).float()
    q = (p / s.double()[..., :, None, :, None]).clamp(-448, 448).float().to(torch.float8_e4m3fn)
    return q.view(*lead, nb * BLOCK, kb * BLOCK)[..., :N, :K].contiguous(), s.contiguous()


def sum_factor(K: int) -> float:
    kb = -(-K // BLOCK)
    return (min(K, BLOCK) + 2 * kb + 2) * STEP


def gemm(xq, xs, wq, ws):
    """(y, bound on the error of the fp32 sum), both fp64."""
    x, w = row_values(xq, xs), weight_values(wq, ws)
    return x @ w.t(), (x.abs() @ w.abs().t()) * sum_factor(x.shape[1])


def swiglu(x, wg, wu, wd):
    """The expert FFN on rows x (fp64 values of quantised rows) with weights in fp64:
    (o, bound on |error of o| before o is weighted or stored)."""
    K, I = wg.shape[1], wg.shape[0]
    f = sum_factor(K)
    g, u = x @ wg.t(), x @ wu.t()
    dg, du = (x.abs() @ wg.abs().t()) * f, (x.abs() @ wu.abs().t()) * f
    sg = torch.sigmoid(g)
    silu = g * sg
    # |silu'| <= 1.1; fast exponential and quotient: (|g| 2^-23 + 2^-21) of silu, and the product
    h = silu * u
    dh = 1.1 * dg * (u.abs() + du) + silu.abs() * du + h.abs() * (g.abs() * 2.0 ** -23 + 2.0 ** -21)
    ph, pd = pad_blocks(h), pad_blocks(dh)
    a = ph.abs().amax(-1, keepdim=True).clamp_min(2.0 ** -100)
    da = pd.amax(-1, keepdim=True)
    v = 448.0 * ph / a
    dv = 448.0 * pd / a + v.abs() * (da / a + 4 * STEP)
    gap, step = e4m3_midpoint_gap(v)
    q = e4m3_round(v)
    # a code can differ by one step where v is within dv of a midpoint (dv is far below a step)
    near = torch.where(gap <= dv, step, 0.0)
    s = a / 448.0
    hv = (q * s).flatten(-2)[:, :I]
    dhv = (near * s + q.abs() * s * (da / a + 2 * STEP)).flatten(-2)[:, :I]
    o = hv @ wd.t()
    return o, dhv @ wd.abs().t() + (hv.abs() @ wd.abs().t()) * sum_factor(I)


def route(z, rule, k, bias=None):
    """Reference routing of one row (numpy fp64 logits): ids, weights, scores."""
    E = len(z)
    off = np.isneginf(z) | np.isnan(z)
    if rule.score == "sigmoid":
        s = np.array([0.0 if o else 1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0
                      for v, o in zip(z, off)])
    else:
        s = np.zeros(E)
        if not off.all():
            m = z[~off].max()
            a = np.where(z[~off] == m, 1.0, np.exp(z[~off] - m))
            s[~off] = a / a.sum()
    val = s + (0.0 if bias is None else bias)
    # order of the choice: (masked class, -key, id); without a bias the logits order it
    cls = np.where(np.isnan(z), 2, np.where(off, 1, 0))
    by = val if bias is not None else z
    gs = E // rule.n_groups
    ranked = []
    for g in range(rule.n_groups):
        ids = [e for e in range(g * gs, (g + 1) * gs) if not off[e]]
        if not ids:
            ranked.append((math.inf, g))
        elif rule.group_score == "top2":
            ranked.append((-sum(sorted((val[e] for e in ids), reverse=True)[:2]), g))
        else:
            ranked.append((-max(by[e] for e in ids), g))
    groups = [g for _, g in sorted(ranked)[:rule.top_groups]] if rule.n_groups > 1 else [0]
    order = sorted((cls[e], 0.0 if cls[e] else -by[e], e)
                   for g in groups for e in range(g * gs, (g + 1) * gs))
    ids = np.array([e for _, _, e in order[:k]], np.int32)
    w = s[ids]
    if rule.renormalize:
        w = w / w.sum() if w.sum() > 0 else w * 0.0
    return ids, w * rule.scale, s[ids]
