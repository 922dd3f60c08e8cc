"""The int8 product, the norm and the int8 codes of rows at the ends of their ranges: sums past
24 bits, rows past fp32, long rows, no rows at all."""
from __future__ import annotations

import pytest
import torch

from sparse_moe_layer_row_gb300 import moe_block as mb
from tests import fp8_ref as F
from tests.test_gpu_rows8 import NORM_ERR, check, outputs

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    mb.load()


def randn(*shape, seed=0, sigma=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda") * sigma


# ----------------------------------------------------------------------- int8 product

def codes(n, K, lo, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(lo, 128, (n, K), generator=g, device="cuda").to(torch.int8)


def product(xq, xs, wq, ws, dt=FP):
    R, K = xq.shape
    N = wq.shape[0]
    mem = torch.zeros(mb.moe_i8_gemm_workspace_bytes(R, N, K), dtype=torch.uint8, device="cuda")
    y = torch.full((R, N), float("nan"), dtype=dt, device="cuda")
    mb.moe_i8_gemm(xq, xs, wq, ws, y, mem)
    torch.cuda.synchronize()
    assert not any(mb.moe_read_device_status(mem).values())
    return y


# few rows, two and four tiles of rows; then the tiles in their three widths with either operand the
# smaller one; K of one and of more parts of 8192, whole and not
SUMS = [(7, 40, 16384), (12, 40, 16384), (200, 40, 16384), (25, 40, (1 << 17) - 16), (40, 300, 1040), (12, 300, 2064),
        (700, 2048, 1024), (2048, 700, 2048), (2048, 701, 2064), (1000, 500, 4096), (264, 2500, 7168),
        (1900, 2100, 2304), (520, 520, 8208), (700, 2048, 8192), (2048, 700, 8208), (2100, 1900, 16400), (300, 2048, (1 << 17) - 16)]


@pytest.mark.parametrize("lo", [100, 127, -128])
@pytest.mark.parametrize("R,N,K", SUMS)
def test_product_sums_past_24_bits(R, N, K, lo):
    """Few rows: the whole number, rounded to fp32 once.  Tiles: each of the K / 16 additions to an
    accumulator and each addition of the parts of 8192 a step of the magnitudes at most, and none where
    no partial sum can pass 2^24; then one rounding."""
    xq, wq = codes(R, K, lo, R), codes(N, K, lo, N + 1)
    if lo == -128:
        xq[:, ::3], wq[:, ::3] = -128, -128
    one = torch.ones(max(R, N), device="cuda")
    y = product(xq, one[:R], wq, one[:N])
    acc = xq.double() @ wq.double().t()   # below 2^53: exact
    mag = xq.double().abs() @ wq.double().abs().t()
    if mb.moe_i8_gemm_workspace_bytes(R, N, K) == 1024 or mag.max() <= 2 ** 24:
        assert torch.equal(y, acc.float())
    else:
        n = min(K, 8192) // 16 + -(-K // 8192)
        assert torch.all((y.double() - acc).abs() <= n * 2.0 ** -23 * mag + 2.0 ** -24 * acc.abs())


@pytest.mark.parametrize("R", [7, 12, 25])
def test_product_of_shares_that_just_pass_24_bits(R):
    """Four warps' shares add up to 2^24, the next ones are 1 and 1, which fp32 drops one after the other."""
    K, N = 2048, 40
    xq, wq = torch.zeros(R, K, dtype=torch.int8, device="cuda"), torch.zeros(N, K, dtype=torch.int8, device="cuda")
    for b in range(16):   # blocks of 128: warp b % 8's
        at = slice(128 * b, 128 * b + (128 if b % 8 < 4 else 1))
        v = -128 if b % 8 < 4 else 1 if b in (4, 5) else 0
        xq[:, at], wq[:, at] = v, v
    one = torch.ones(N, device="cuda")
    acc = xq.double() @ wq.double().t()
    assert torch.all(acc == 2 ** 24 + 2)
    assert torch.equal(product(xq, one[:R], wq, one).double(), acc)


def test_product_row_does_not_depend_on_its_batch():
    """The same bits alone, with a few rows and among many: past 24 bits on the kernel for few rows,
    below on both."""
    for N, K, rows in ((600, 2304, (1, 8, 9, 16, 17, 33)), (2048, 1024, (1, 8, 9, 17, 130, 600, 1000))):
        xq, wq = codes(1000, K, 100, 1), codes(N, K, 100, 2)
        xs, ws = torch.exp(randn(1000, seed=3)) * 0.01, torch.exp(randn(N, seed=4)) * 0.01
        for dt in (BF, FP):
            y = product(xq[:rows[-1]], xs[:rows[-1]], wq, ws, dt)
            for R in rows:
                assert torch.equal(product(xq[:R], xs[:R], wq, ws, dt), y[:R])


# ----------------------------------------------------------------- rows beyond fp32

def huge_rows(R, H, dt, seed=1):
    """Ordinary rows, whose sum of squares a block of 1e25 takes past fp32, with a block of tiny values."""
    x = randn(R, H, seed=seed)
    x[:, :min(128, H // 3)] = 1e25 * (1 + randn(R, min(128, H // 3), seed=seed + 1).abs())
    x[:, 2 * H // 3:] *= 1e-8
    return x.to(dt)


def check_far(r, w, eps, dt, y, codes, scales):
    """test_gpu_rows8's check, with scales that may lie below fp32's normal range: the product with rstd
    and the quotient are rounded to steps of 2^-149 there."""
    if codes is not None:
        p = r.double() * (1.0 if w is None else w.double())
        rstd = torch.rsqrt(r.double().square().mean(1, keepdim=True) + eps)
        if codes.dtype == torch.int8:
            s = (p.abs().amax(1, keepdim=True).clamp_min(2.0 ** -100) * rstd / 127.0)[:, 0]
        else:
            s = (F.pad_blocks(p).abs().amax(-1).clamp_min(2.0 ** -100) * rstd / 448.0).t()
        assert torch.all((scales.double() - s).abs() <= 2 * NORM_ERR * s + 2 * 2.0 ** -149)
        scales = s
    check(r, w, eps, dt, y, codes, scales)


# a row per CTA, rows of CTAs that stay, unaligned rows, rows that are read twice
HUGE = [(3, 2048), (700, 200), (700, 2048), (700, 7168), (5, 1001), (2, 40000), (2, 33001)]


@pytest.mark.parametrize("dt", [BF, FP], ids=str)
@pytest.mark.parametrize("R,H", HUGE)
def test_norm_codes_of_rows_beyond_fp32(R, H, dt):
    """Codes do not depend on the sum of squares: they are those of the plain quantising calls."""
    x = huge_rows(R, H, dt)
    want, ws = torch.empty(R, H, dtype=E4M3, device="cuda"), torch.empty(-(-H // 128), R, device="cuda")
    mb.moe_fp8_quantize(x, want, ws)
    want8, ws8 = torch.empty(R, H, dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
    mb.moe_i8_quantize(x, want8, ws8)
    for res in (None, torch.zeros(R, H, dtype=dt, device="cuda"), torch.zeros(R, H, device="cuda")):
        for total in ((None,) if res is None else (None, torch.empty_like(res))):
            y, q, s = outputs(R, H, dt, "y+e4m3")
            mb.moe_add_rmsnorm(x, None, 1e-6, residual=res, total=total, y=y, codes=q, scales=s)
            assert torch.equal(q.view(torch.uint8), want.view(torch.uint8))
            check_far(x, None, 1e-6, dt, y, q, s)
            y, q, s = outputs(R, H, dt, "y+i8")
            mb.moe_add_rmsnorm(x, None, 1e-6, residual=res, total=total, y=y, codes=q, scales=s)
            assert torch.equal(q, want8)
            check_far(x, None, 1e-6, dt, y, q, s)
    if dt == FP:   # the sum is formed again from what is not overwritten yet
        y, q, s = outputs(R, H, dt, "y+i8")
        at = x.clone()
        mb.moe_add_rmsnorm(at, None, 1e-6, residual=torch.zeros_like(x), y=at, codes=q, scales=s)
        check_far(x, None, 1e-6, dt, at, q, s)


@pytest.mark.parametrize("R,H", HUGE)
def test_norm_products_beyond_fp32(R, H):
    """r w passes fp32: such blocks (int8: rows) are scaled; the others' codes are those of r w."""
    x = huge_rows(R, H, FP)
    x[:, 1] = 3e38
    w = 1 + 0.2 * randn(H, seed=5)
    w[:4] = 4.0
    for out in ("y+e4m3", "y+i8", "y"):
        y, q, s = outputs(R, H, FP, out)
        mb.moe_add_rmsnorm(x, w, 1e-6, y=y, codes=q, scales=s)
        check_far(x, w, 1e-6, FP, y, q, s)
        assert torch.isfinite(y).all()


@pytest.mark.parametrize("R,H", [(400, 8192), (2, 8192), (2, 1 << 16), (2, (1 << 16) + 1)])
def test_norm_eps_of_rows_beyond_fp32(R, H):
    """The largest eps counts beside a sum of squares just beyond fp32."""
    x = randn(R, H, seed=3).sign() * (2.0 ** 128.2 / H) ** 0.5
    y, q, s = outputs(R, H, FP, "y+i8")
    mb.moe_add_rmsnorm(x, None, 2.0 ** 100, y=y, codes=q, scales=s)
    check_far(x, None, 2.0 ** 100, FP, y, q, s)


# ------------------------------------------------------------------------- long rows

@pytest.mark.parametrize("scale", [1.0, 2.0 ** 70])
@pytest.mark.parametrize("H", [1 << 20, (1 << 22) + 8, (1 << 22) + 3, 1 << 26])
def test_norm_of_long_rows(H, scale):
    """Rows of equal values, whose serial sum would lose bits, hold the bound of short ones."""
    for dt in (FP, BF):
        x = torch.full((1, H), 1.1 * scale, dtype=dt, device="cuda")
        x[0, ::3] *= -1
        y, _, _ = outputs(1, H, dt, "y")
        mb.moe_add_rmsnorm(x, None, 1e-6, y=y)
        check(x, None, 1e-6, dt, y, None, None)


# --------------------------------------------------------------------------- no rows

def test_calls_of_no_rows():
    """An empty batch: tensors of no rows, whose pointers are null, are taken by every call."""
    x = torch.empty(0, 256, dtype=BF, device="cuda")
    res = torch.empty(0, 256, device="cuda")
    for out in ("y", "e4m3", "i8", "y+e4m3", "y+i8"):
        for r in (None, x.clone(), res):
            y, q, s = outputs(0, 256, BF, out)
            mb.moe_add_rmsnorm(x, None, 1e-6, residual=r, total=r, y=y, codes=q, scales=s)
    _, q, s = outputs(0, 256, BF, "i8")
    mb.moe_i8_quantize(x, q, s)
    wq, ws = codes(40, 256, -128, 1), torch.ones(40, device="cuda")
    mb.moe_i8_gemm(q, s, wq, ws, torch.empty(0, 40, device="cuda"), torch.zeros(1024, dtype=torch.uint8, device="cuda"))


# -------------------------------------------------------------------------- wait limit

@pytest.mark.parametrize("R,N,K", [(700, 2048, 336), (2048, 700, 2064), (2100, 1900, 16400), (300, 2048, 8208)])
def test_product_wait_limit(R, N, K):
    """With a limit of 1 ns the tiles' waits run out: the call returns and counts them, one for a warp
    that waits at most, and the next call, on the same workspace, is right bit for bit."""
    xq, wq = codes(R, K, -128, 1), codes(N, K, -128, 2)
    one = torch.ones(max(R, N), device="cuda")
    mem = torch.zeros(mb.moe_i8_gemm_workspace_bytes(R, N, K), dtype=torch.uint8, device="cuda")
    assert mem.numel() > 2 * K * min(R, N)
    y, want = torch.empty(R, N, device="cuda"), torch.empty(R, N, device="cuda")
    mb.moe_i8_gemm(xq, one[:R], wq, one[:N], want, mem)
    torch.cuda.synchronize()
    assert not any(mb.moe_read_device_status(mem).values())
    for _ in range(3):
        mb.moe_i8_gemm_set_wait_limit(1)
        try:
            mb.moe_i8_gemm(xq, one[:R], wq, one[:N], y, mem)
            torch.cuda.synchronize()
        finally:
            mb.moe_i8_gemm_set_wait_limit(0)
        st = mb.moe_read_device_status(mem)
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        assert 0 < st["wait_timeout"] <= 16 * sms, st
        mb.moe_clear_device_status(mem)
        y.fill_(float("nan"))
        mb.moe_i8_gemm(xq, one[:R], wq, one[:N], y, mem)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and not any(mb.moe_read_device_status(mem).values())


# --------------------------------------------------------------------------- refusals

def test_arguments_that_are_no_tensors_are_named():
    x = randn(4, 256).to(BF)
    s, q, w = torch.empty(4, device="cuda"), torch.empty(4, 256, dtype=torch.int8, device="cuda"), torch.empty(0)
    for kw, word in ((dict(codes=[1], scales=s), "codes"), (dict(codes=q, scales=[1.0]), "scales"), (dict(y="y"), "y"),
                     (dict(y=x.clone(), residual=1.0), "residual"), (dict(y=x.clone(), residual=x, total=3), "total")):
        with pytest.raises(TypeError, match=word):
            mb.moe_add_rmsnorm(x, None, 1e-6, **kw)
    with pytest.raises(TypeError, match="weight"):
        mb.moe_add_rmsnorm(x, 1.0, 1e-6, y=x.clone())
    for args, word in (((None, s, q, s, x, w), "xq"), ((q, None, q, s, x, w), "xs"), ((q, s, 1, s, x, w), "wq")):
        with pytest.raises(TypeError, match=word):
            mb.moe_i8_gemm(*args)
    with pytest.raises(TypeError, match="codes"):
        mb.moe_i8_quantize(x, None, s)
