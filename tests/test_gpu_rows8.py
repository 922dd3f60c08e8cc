"""The residual norm, the int8 codes of rows and the int8 product against plain 64-bit references.

Bounds.  A sum of squares of H values is off by at most (values per thread + steps of the
tree) 2^-24 of itself, below 64 x 2^-24 at the sizes here; rstd carries half of that and
three roundings, p and p rstd one each: below 2^-18 of the value in all.
"""
from __future__ import annotations

import pytest
import torch

from sparse_moe_layer_row_gb300 import moe_block as mb
from tests import fp8_ref as F

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
NORM_ERR = 2.0 ** -18
TINY = {BF: 2.0 ** -133, HF: 2.0 ** -24, FP: 2.0 ** -149}   # a type's least step


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    mb.load()


def randn(*shape, seed=0, sigma=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda") * sigma


# ------------------------------------------------------------------------------ norm

def outputs(R, H, dt, out):
    y = torch.full((R, H), float("nan"), dtype=dt, device="cuda") if out in ("y", "y+i8", "y+e4m3") else None
    codes = scales = None
    if "i8" in out:
        codes = torch.zeros(R, H, dtype=torch.int8, device="cuda")
        scales = torch.full((R,), float("nan"), device="cuda")
    elif "e4m3" in out:
        codes = torch.zeros(R, H, dtype=torch.uint8, device="cuda").view(E4M3)
        scales = torch.full((-(-H // 128), R), float("nan"), device="cuda")
    return y, codes, scales


def check(r, w, eps, dt, y, codes, scales):
    """Outputs against the norm of r (the stored sum) in 64 bits."""
    r = r.double()
    R, H = r.shape
    wd = torch.ones(H, dtype=torch.float64, device="cuda") if w is None else w.double()
    p = r * wd
    rstd = torch.rsqrt(r.square().mean(1, keepdim=True) + eps)
    v = p * rstd
    if y is not None:
        bound = (F.HALF[dt] * (1 + NORM_ERR) + NORM_ERR) * v.abs() + TINY[dt]
        assert torch.all((y.double() - v).abs() <= bound)
    if codes is None:
        return
    if codes.dtype == torch.int8:
        a = p.abs().amax(1, keepdim=True).clamp_min(2.0 ** -100)
        q = 127.0 * p / a
        # two roundings before the code's, and p's own
        near = ((q.abs() % 1.0) - 0.5).abs() <= 4 * F.STEP * q.abs()
        assert torch.all((codes.double() == q.round()) | (near & ((codes.double() - q).abs() <= 0.5 + 1e-4)))
        s = (a * rstd)[:, 0] / 127.0
    else:
        pb = F.pad_blocks(p)
        a = pb.abs().amax(-1, keepdim=True).clamp_min(2.0 ** -100)
        q = (448.0 * pb / a).view(R, -1)[:, :H]
        gap, step = F.e4m3_midpoint_gap(q)
        near = gap <= 4 * F.STEP * q.abs()
        assert torch.all((codes.double() == F.e4m3_round(q)) | (near & ((codes.double() - q).abs() <= step)))
        s = (a[..., 0] * rstd / 448.0).t()
    assert torch.all((scales.double() - s).abs() <= 2 * NORM_ERR * s)


def residual_sum(x, res, total):
    """total against x + residual: rounded to fp32 and to its type."""
    s = x.double() + res.double()
    assert torch.all((total.double() - s).abs() <= (F.HALF[total.dtype] + 2.0 ** -23) * s.abs() + TINY[total.dtype])


SHAPES = [(1, 2048), (1, 1), (3, 7), (5, 1000), (70, 136), (700, 2048), (2000, 520), (2, 16384), (1300, 264), (2, 40000), (3, 33001)]


@pytest.mark.parametrize("out", ["y", "e4m3", "i8", "y+i8", "y+e4m3"])
@pytest.mark.parametrize("dt,rt,wt", [(BF, BF, BF), (BF, FP, FP), (HF, HF, FP), (FP, FP, FP), (BF, None, BF), (FP, None, None)], ids=str)
def test_norm(dt, rt, wt, out):
    for i, (R, H) in enumerate(SHAPES):
        x = (randn(R, H, seed=i) * torch.exp(randn(R, 1, seed=i + 50))).to(dt)
        res = None if rt is None else randn(R, H, seed=i + 100, sigma=3.0).to(rt)
        w = None if wt is None else (1 + 0.2 * randn(H, seed=i + 150)).to(wt)
        total = None if rt is None else torch.full((R, H), float("nan"), dtype=rt, device="cuda")
        y, codes, scales = outputs(R, H, dt, out)
        mb.moe_add_rmsnorm(x, w, 1e-5, residual=res, total=total, y=y, codes=codes, scales=scales)
        torch.cuda.synchronize()
        if rt is not None:
            residual_sum(x, res, total)
        check(x if rt is None else total, w, 1e-5, dt, y, codes, scales)
        if rt is not None:   # the same without the sum's store, and in place
            y2, c2, s2 = outputs(R, H, dt, out)
            mb.moe_add_rmsnorm(x, w, 1e-5, residual=res, y=y2, codes=c2, scales=s2)
            y3, c3, s3 = outputs(R, H, dt, out)
            inplace = res.clone()
            mb.moe_add_rmsnorm(x, w, 1e-5, residual=inplace, total=inplace, y=y3, codes=c3, scales=s3)
            assert torch.equal(inplace, total)
            for a, b, c in ((y, y2, y3), (codes, c2, c3), (scales, s2, s3)):
                if a is not None:
                    a, b, c = (t.float() for t in (a, b, c))
                    assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("H", [2048, 1000, 40000])
def test_norm_in_place_of_x(H):
    x, res = randn(4, H, seed=1).to(BF), randn(4, H, seed=2).to(BF)
    total, y = torch.empty_like(x), torch.empty_like(x)
    mb.moe_add_rmsnorm(x, None, 1e-6, residual=res, total=total, y=y)
    xt = x.clone()
    y2 = torch.empty_like(x)
    mb.moe_add_rmsnorm(xt, None, 1e-6, residual=res, total=xt, y=y2)
    xy = x.clone()
    mb.moe_add_rmsnorm(xy, None, 1e-6, residual=res, y=xy)
    assert torch.equal(xt, total) and torch.equal(y2, y) and torch.equal(xy, y)


@pytest.mark.parametrize("H", [8, 248, 256, 264, 512, 776, 2048, 4096, 4104, 8192, 8200, 32768, 32776])
@pytest.mark.parametrize("dt,rt", [(BF, BF), (BF, FP), (HF, HF), (FP, FP)], ids=str)
def test_norm_many_rows_in_place(dt, rt, H):
    """More rows than CTAs, whose next row is loaded while one is worked on: in place gives what
    separate buffers give, at the edges of the kernels' widths; rows and columns beyond stay."""
    R = 1400 if H <= 8200 else 320
    x, res = randn(R, H, seed=H).to(dt), randn(R, H, seed=H + 1).to(rt)
    w = (1 + 0.2 * randn(H, seed=H + 2)).to(rt)
    total = torch.empty_like(res)
    y, q, s = outputs(R, H, dt, "y+i8")
    mb.moe_add_rmsnorm(x, w, 1e-6, residual=res, total=total, y=y, codes=q, scales=s)
    residual_sum(x, res, total)
    check(total, w, 1e-6, dt, y, q, s)
    _, q2, s2 = outputs(R, H, dt, "y+i8")
    rbuf = torch.full((R + 2, H), 9.0, dtype=rt, device="cuda")
    rbuf[:R] = res
    xbuf = torch.full((R + 2, H), 9.0, dtype=dt, device="cuda")
    xbuf[:R] = x
    mb.moe_add_rmsnorm(xbuf[:R], w, 1e-6, residual=rbuf[:R], total=rbuf[:R], y=xbuf[:R], codes=q2, scales=s2)
    assert torch.equal(rbuf[:R], total) and torch.equal(xbuf[:R], y) and torch.equal(q2, q) and torch.equal(s2, s)
    assert torch.all(rbuf[R:] == 9) and torch.all(xbuf[R:] == 9)
    if rt == dt:   # the sum in x's place
        xt = x.clone()
        y3, _, _ = outputs(R, H, dt, "y")
        mb.moe_add_rmsnorm(xt, w, 1e-6, residual=res, total=xt, y=y3)
        assert torch.equal(xt, total) and torch.equal(y3, y)


def test_norm_codes_are_those_of_the_plain_formula():
    """Bit for bit: codes are formed from the stored sum by the stated fp32 operations."""
    for dt, H in ((BF, 2048), (FP, 1000), (HF, 640)):
        x, res, w = randn(300, H, seed=3).to(dt), randn(300, H, seed=4).to(dt), (1 + 0.1 * randn(H, seed=5)).to(dt)
        total = torch.empty_like(x)
        _, q8, s8 = outputs(300, H, dt, "i8")
        mb.moe_add_rmsnorm(x, w, 1e-6, residual=res, total=total, codes=q8, scales=s8)
        _, qf, sf = outputs(300, H, dt, "e4m3")
        mb.moe_add_rmsnorm(x, w, 1e-6, residual=res, codes=qf, scales=sf)
        p = total.float() * w.float()
        a = p.abs().amax(1, keepdim=True)
        assert torch.equal((p * (127 / 128) / (a * 2.0 ** -7)).round().to(torch.int8), q8)
        pb = F.pad_blocks(p)
        v = pb * 0.875 / (pb.abs().amax(-1, keepdim=True).clamp_min(2.0 ** -100) * 2.0 ** -9)
        assert torch.equal(v.to(E4M3).view(torch.uint8).view(300, -1)[:, :H], qf.view(torch.uint8))


def test_norm_strided_rows():
    wide = randn(40, 3000, seed=2).to(BF)
    ybuf = torch.full((40, 700), float("nan"), dtype=BF, device="cuda")
    for c0, H in ((0, 512), (8, 512), (3, 512), (1, 131)):
        x, res = wide[:, c0:c0 + H], wide[:, 1000 + c0:1000 + c0 + H]
        want, total = torch.empty(40, H, dtype=BF, device="cuda"), torch.empty(40, H, dtype=BF, device="cuda")
        mb.moe_add_rmsnorm(x.contiguous(), None, 1e-6, residual=res.contiguous(), total=total, y=want)
        ybuf.fill_(float("nan"))
        tbuf = torch.full((40, 600), float("nan"), dtype=BF, device="cuda")
        y, t = ybuf[:, c0:c0 + H], tbuf[:, 2:2 + H]
        mb.moe_add_rmsnorm(x, None, 1e-6, residual=res, total=t, y=y)
        # (another number of threads may hold the row: the sums' last bits differ)
        check(t, None, 1e-6, BF, y, None, None)
        assert torch.equal(t, total) and torch.all((y.float() - want.float()).abs() <= 2 ** -7 * want.float().abs())
        outside = torch.ones(700, dtype=torch.bool, device="cuda")
        outside[c0:c0 + H] = False
        assert torch.isnan(ybuf[:, outside]).all() and torch.isnan(tbuf[:, :2]).all() and torch.isnan(tbuf[:, 2 + H:]).all()


def test_norm_zero_huge_tiny_and_nonfinite_rows():
    H = 1024
    for dt in (FP, BF):
        x = randn(8, H, seed=6)
        x[0] = 0.0
        x[1] *= 2.0 ** 100          # the sum of squares exceeds fp32
        x[2] *= 2.0 ** -80
        x[3, 5] = 3e38
        x = x.to(dt)
        y, q, s = outputs(8, H, dt, "y+i8")
        mb.moe_add_rmsnorm(x, None, 1e-6, y=y, codes=q, scales=s)
        check(x[:4], None, 1e-6, dt, y[:4], q[:4], s[:4])
        yf, qf, sf = outputs(8, H, dt, "y+e4m3")
        mb.moe_add_rmsnorm(x, None, 1e-6, y=yf, codes=qf, scales=sf)
        check(x[:4], None, 1e-6, dt, yf[:4], qf[:4], sf[:4, :4] if sf.shape[0] == 4 else sf[:, :4])
        x[4, 3], x[5, 7], x[6, 1000] = float("nan"), float("inf"), float("-inf")
        for out in ("y+i8", "y+e4m3"):
            y2, q2, s2 = outputs(8, H, dt, out)
            mb.moe_add_rmsnorm(x, None, 1e-6, y=y2, codes=q2, scales=s2)
            base, qb, sb = (y, q, s) if out == "y+i8" else (yf, qf, sf)
            clean = torch.tensor([0, 1, 2, 3, 7], device="cuda")
            assert torch.equal(y2[clean], base[clean]) and torch.equal(q2[clean].float(), qb[clean].float())
            assert torch.isnan(y2[4]).all() and torch.isnan(y2[5, 7]) and torch.isnan(y2[6, 1000])
            if out == "y+i8":
                assert torch.isnan(s2[4:7]).all() and torch.equal(s2[clean], sb[clean])
            else:
                assert torch.isnan(s2[:, 4]).all() and torch.isnan(s2[0, 5]) and torch.isnan(s2[7, 6])


def test_norm_stream_graph_and_rows_behind():
    x, res = randn(33, 2048, seed=8).to(BF), randn(33, 2048, seed=9).to(BF)
    want, twant = torch.empty_like(x), torch.empty_like(x)
    mb.moe_add_rmsnorm(x, None, 1e-6, residual=res, total=twant, y=want)
    big = torch.full((40, 2048), 7.0, dtype=BF, device="cuda")
    tot = torch.empty_like(x)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    mb.moe_add_rmsnorm(x, None, 1e-6, residual=res, total=tot, y=big[:33], stream=st)
    st.synchronize()
    assert torch.equal(big[:33], want) and torch.equal(tot, twant) and torch.all(big[33:] == 7)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        mb.moe_add_rmsnorm(x, None, 1e-6, residual=res, total=tot, y=big[:33], stream=st)
    x.copy_(randn(33, 2048, seed=10).to(BF))
    g.replay()
    torch.cuda.synchronize()
    mb.moe_add_rmsnorm(x, None, 1e-6, residual=res, total=twant, y=want)
    assert torch.equal(big[:33], want) and torch.equal(tot, twant)


def test_norm_binding_refuses():
    x = randn(4, 256, seed=1).to(BF)
    y, q = torch.empty_like(x), torch.empty(4, 256, dtype=torch.int8, device="cuda")
    s = torch.empty(4, device="cuda")
    w = torch.ones(256, dtype=BF, device="cuda")
    bad = [dict(y=y.half()), dict(y=y, residual=x.half()), dict(y=y, residual=x, total=x.float()),
           dict(y=y, total=x.clone()), dict(codes=q), dict(codes=q, scales=s[:3]), dict(scales=s, y=y),
           dict(y=y[:3]), dict(codes=q.view(torch.uint8), scales=s), dict(y=y, weight=w.half()), dict(y=y, weight=w[:255])]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            mb.moe_add_rmsnorm(x, kw.pop("weight", w), 1e-6, **kw)
    with pytest.raises(mb.MoeError):
        mb.moe_add_rmsnorm(x, w, 1e-6)
    with pytest.raises(mb.MoeError):
        mb.moe_add_rmsnorm(x, w, 0.0, y=y)


# -------------------------------------------------------------------- int8 quantising

def quantize(x):
    q = torch.full(x.shape, 99, dtype=torch.int8, device="cuda")
    s = torch.full((x.shape[0],), float("nan"), device="cuda")
    mb.moe_i8_quantize(x, q, s)
    torch.cuda.synchronize()
    return q, s


@pytest.mark.parametrize("dt", [BF, HF, FP], ids=str)
@pytest.mark.parametrize("R,K", [(1, 128), (1, 1), (3, 7), (32, 2048), (5, 1000), (700, 136), (257, 640), (2, 4104), (2, 33000), (2, 33003)])
def test_quantize(R, K, dt):
    x = (randn(R, K, seed=R + K) * torch.exp(2 * randn(R, 1, seed=7))).to(dt)
    q, s = quantize(x)
    xd = x.double()
    a = xd.abs().amax(1, keepdim=True).clamp_min(2.0 ** -100)
    assert torch.equal(s, (a[:, 0] / 127.0).float())
    v = 127.0 * xd / a
    if dt == FP:
        near = ((v.abs() % 1.0) - 0.5).abs() <= 2 * F.STEP * v.abs()
        assert torch.all((q.double() == v.round()) | near)
        p = x * (127 / 128) / (x.abs().amax(1, keepdim=True) * 2.0 ** -7)
        assert torch.equal(q, p.round().to(torch.int8))
    else:
        assert torch.equal(q.double(), v.round())


def test_quantize_ties_tiny_huge_and_nonfinite():
    x = torch.zeros(8, 512, device="cuda")
    x[0, 0] = 127.0
    x[0, 1:128] = torch.arange(127, device="cuda") + 0.5
    x[1] = -x[0] * 2.0 ** 60
    x[2] = 1e-38
    x[3, 5] = torch.finfo(FP).max
    x[3, 6] = -torch.finfo(FP).max / 3
    x[4, 511] = -2.0 ** -120
    ok = x.clone()
    x[5, 1], x[6, 3], x[7, 9] = float("nan"), float("inf"), float("-inf")
    x[7, 10] = float("nan")
    q, s = quantize(x)
    a = ok.double().abs().amax(1, keepdim=True).clamp_min(2.0 ** -100)
    assert torch.equal(q[:5].double(), (127 * ok.double() / a).round()[:5])
    assert torch.equal(s[:5], (a[:, 0] / 127).float()[:5])
    assert torch.isnan(q[5:].float() * s[5:, None]).all()


def test_quantize_strided():
    wide = randn(40, 700, seed=2).to(BF)
    for c0, K in ((0, 512), (8, 512), (3, 512), (1, 130)):
        q, s = quantize(wide[:, c0:c0 + K])
        q2, s2 = quantize(wide[:, c0:c0 + K].contiguous())
        assert torch.equal(q, q2) and torch.equal(s, s2)


# ----------------------------------------------------------------------- int8 product

def codes(*shape, seed, full=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if full:
        return torch.randint(-128, 128, shape, generator=g, device="cuda").to(torch.int8)
    return (torch.randn(*shape, generator=g, device="cuda") * 35).clamp(-127, 127).round().to(torch.int8)


def product(xq, xs, wq, ws, dt=FP, y=None):
    R, K = xq.shape
    N = wq.shape[0]
    mem = torch.zeros(mb.moe_i8_gemm_workspace_bytes(R, N, K), dtype=torch.uint8, device="cuda")
    if y is None:
        y = torch.full((R, N), float("nan"), dtype=dt, device="cuda")
    mb.moe_i8_gemm(xq, xs, wq, ws, y, mem)
    torch.cuda.synchronize()
    assert not any(mb.moe_read_device_status(mem).values())
    return y


def reference(xq, xs, wq, ws):
    """The sum (whole numbers, exact in 64 bits) and its scale in fp32."""
    acc = xq.double() @ wq.double().t()
    return acc, (xs[:, None] * ws).double(), xq.double().abs() @ wq.double().abs().t()


GEMMS = [(1, 1, 16), (1, 2048, 2048), (3, 40, 48), (8, 129, 1104), (17, 1000, 272), (32, 256, 4096), (33, 64, 128),
         (77, 1000, 1104), (128, 128, 128), (130, 513, 2064), (300, 2048, 512), (257, 1, 80), (1000, 777, 2048), (64, 4096, 7168)]


@pytest.mark.parametrize("dt", [BF, HF, FP], ids=str)
@pytest.mark.parametrize("R,N,K", GEMMS)
def test_product(R, N, K, dt):
    xq, wq = codes(R, K, seed=R), codes(N, K, seed=N + 1)
    xs, ws = torch.exp(randn(R, seed=2)) * 0.01, torch.exp(randn(N, seed=3)) * 0.003
    y = product(xq, xs, wq, ws, dt)
    acc, sc, mag = reference(xq, xs, wq, ws)
    # sums of whole numbers below 2^24 are exact; else each addition a step of the magnitudes
    off = torch.where(mag < 2 ** 24, 0.0, mag * K * F.STEP)
    v = acc * sc
    assert torch.all((y.double() - v).abs() <= (F.HALF[dt] + 2.0 ** -24) * v.abs() + off * sc + TINY[dt])


# tiles of 64, 128 and 256 rows of the smaller operand, either operand the smaller one; K that ends in
# the first or second half of a stage, or before it; rows of y that begin anywhere
TILES = [(700, 2048, 336), (2048, 700, 336), (2048, 701, 400), (1900, 2100, 400), (2100, 1900, 400), (2100, 1901, 144),
         (300, 2048, 512), (1000, 500, 592), (2000, 2000, 16), (1500, 1510, 80), (9000, 264, 272), (264, 9001, 272)]


@pytest.mark.parametrize("dt", [BF, FP], ids=str)
@pytest.mark.parametrize("R,N,K", TILES)
def test_product_of_tiles(R, N, K, dt):
    assert mb.moe_i8_gemm_workspace_bytes(R, N, K) > 2 * K * min(R, N)
    xq, wq = codes(R, K, seed=R), codes(N, K, seed=N + 1)
    xs, ws = torch.exp(randn(R, seed=2)) * 0.01, torch.exp(randn(N, seed=3)) * 0.003
    y = product(xq, xs, wq, ws, dt)
    acc, sc, mag = reference(xq, xs, wq, ws)
    v = acc * sc
    assert float(mag.max()) < 2 ** 24   # exact sums
    assert torch.all((y.double() - v).abs() <= (F.HALF[dt] + 2.0 ** -24) * v.abs() + TINY[dt])


@pytest.mark.parametrize("R,N,K", [(4, 64, 1024), (40, 300, 1024), (200, 300, 1008), (1030, 520, 960)])
def test_product_of_whole_numbers_is_exact(R, N, K):
    """Any codes, -128 among them, scales 1: whole numbers below 2^24 come out as they are."""
    xq, wq = codes(R, K, seed=1, full=True), codes(N, K, seed=2, full=True)
    xq[:, :8], wq[:, :8] = -128, -128
    one = torch.ones(max(R, N), device="cuda")
    y = product(xq, one[:R], wq, one[:N])
    assert torch.equal(y.double(), xq.double() @ wq.double().t())


@pytest.mark.parametrize("R", [5, 200])
def test_product_beyond_24_bits(R):
    """All codes at their largest and K near its limit: the sum is held in 32 bits."""
    K, N = (1 << 17) - 16, 40
    xq = torch.full((R, K), -128, dtype=torch.int8, device="cuda")
    wq = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    wq[::2] = 127
    wq[1, ::2] = 127
    one = torch.ones(max(R, N), device="cuda")
    y = product(xq, one[:R], wq, one[:N]).double()
    acc = xq.double() @ wq.double().t()
    assert torch.all((y - acc).abs() <= K * F.STEP * (xq.double().abs() @ wq.double().abs().t()))
    assert torch.all((y - acc).abs()[:, [0, 2, 3]] <= 2.0 ** -9 * acc.abs()[:, [0, 2, 3]])


@pytest.mark.parametrize("R,N,K", [(3, 100, 256), (150, 300, 512), (500, 1000, 1040)])
def test_product_strided_output_and_nonfinite_scales(R, N, K):
    xq, wq = codes(R, K, seed=5), codes(N, K, seed=6)
    xs, ws = torch.ones(R, device="cuda"), torch.ones(N, device="cuda")
    for dt in (BF, FP):
        want = product(xq, xs, wq, ws, dt)
        for c0 in (0, 8, 3):
            buf = torch.full((R + 2, N + 16), 5.0, dtype=dt, device="cuda")
            product(xq, xs, wq, ws, y=buf[:R, c0:c0 + N])
            assert torch.equal(buf[:R, c0:c0 + N], want)
            assert torch.all(buf[R:] == 5) and torch.all(buf[:, :c0] == 5) and torch.all(buf[:, c0 + N:] == 5)
    xs[1], ws[2] = float("nan"), float("inf")
    xq[1] = 0
    y = product(xq, xs, wq, ws, FP)
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[:, 2]).any()
    rest = torch.ones(R, N, dtype=torch.bool, device="cuda")
    rest[1], rest[:, 2] = False, False
    assert torch.equal(y[rest], product(xq, torch.ones_like(xs), wq, torch.ones_like(ws))[rest])


@pytest.mark.parametrize("R,N,K", [(6, 500, 528), (30, 500, 528), (600, 2000, 528)])
def test_product_stream_and_graph(R, N, K):
    """On another stream, and captured and replayed on new codes; the workspace's contents and
    what ran before in it do not show."""
    xq, wq = codes(R, K, seed=11), codes(N, K, seed=12)
    xs, ws = torch.exp(randn(R, seed=13)) * 0.01, torch.exp(randn(N, seed=14)) * 0.003
    want = product(xq, xs, wq, ws, BF)
    mem = torch.zeros(mb.moe_i8_gemm_workspace_bytes(R, N, K), dtype=torch.uint8, device="cuda")
    mem[1024:] = 0xFF
    y = torch.full((R + 1, N), 5.0, dtype=BF, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    mb.moe_i8_gemm(xq, xs, wq, ws, y[:R], mem, stream=st)
    st.synchronize()
    assert torch.equal(y[:R], want) and torch.all(y[R:] == 5)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        mb.moe_i8_gemm(xq, xs, wq, ws, y[:R], mem)
    for i in range(5):
        xq.copy_(codes(R, K, seed=20 + i))
        xs.mul_(1.25)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y[:R], product(xq, xs, wq, ws, BF)) and torch.all(y[R:] == 5)
    assert not any(mb.moe_read_device_status(mem).values())


def test_quantize_then_product_back_to_back():
    """Codes and scales written by one call and read by the next, with no wait of the host
    between: a kernel may start before the one ahead of it ends."""
    for R, N, K in ((4, 1000, 2048), (24, 1000, 2048), (1000, 1000, 2048)):
        W, x = randn(N, K, seed=1), [randn(R, K, seed=2 + i).to(BF) for i in range(8)]
        wq, ws = quantize(W)
        mem = torch.zeros(mb.moe_i8_gemm_workspace_bytes(R, N, K), dtype=torch.uint8, device="cuda")
        q, s = torch.empty(R, K, dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
        ys = [torch.empty(R, N, device="cuda") for _ in x]
        for xi, yi in zip(x, ys):
            mb.moe_i8_quantize(xi, q, s)
            mb.moe_i8_gemm(q, s, wq, ws, yi, mem)
        torch.cuda.synchronize()
        for xi, yi in zip(x, ys):
            assert torch.equal(yi, product(*quantize(xi), wq, ws))


def test_norm_codes_feed_both_products():
    """norm + residual -> codes -> product, against the same in 64 bits from the codes."""
    R, H, N = 65, 1024, 384
    x, res, w = randn(R, H, seed=1).to(BF), randn(R, H, seed=2, sigma=3).to(BF), (1 + 0.1 * randn(H, seed=3)).to(BF)
    total = torch.empty_like(x)
    W = randn(N, H, seed=4, sigma=0.02)
    wq, ws = quantize(W)
    _, q, s = outputs(R, H, BF, "i8")
    mb.moe_add_rmsnorm(x, w, 1e-6, residual=res, total=total, codes=q, scales=s)
    y = product(q, s, wq, ws)
    v = total.double() * w.double()
    v = v * torch.rsqrt(total.double().square().mean(1, keepdim=True) + 1e-6)
    full = v @ W.double().t()
    # a code is off by half of 1 / 127 of its row's largest value, on either side
    dx, dw = s.double()[:, None] * 0.5, ws.double()[None, :] * 0.5
    bound = dx * W.double().abs().sum(1) + v.abs().sum(1, keepdim=True) * dw + H * dx * dw
    assert torch.all((y.double() - full).abs() <= bound * 1.001)
    wf, wfs = F.block_codes(W)
    _, qf, sf = outputs(R, H, BF, "e4m3")
    mb.moe_add_rmsnorm(x, w, 1e-6, residual=res, codes=qf, scales=sf)
    mem = torch.zeros(mb.moe_fp8_gemm_workspace_bytes(R, N, H), dtype=torch.uint8, device="cuda")
    yf = torch.empty(R, N, device="cuda")
    mb.moe_fp8_gemm(qf, sf, wf, wfs, yf, mem)
    ref, bound = F.gemm(qf, sf, wf, wfs)
    assert torch.all((yf.double() - ref).abs() <= bound)
