"""The int8 product, the norm and the int8 codes of rows at the ends of their ranges: sums past
24 bits, rows past fp32, long rows, no rows at all."""
from __future__ import annotations

import pytest
import torch

from sparse_moe_layer_row_gb300 import moe_block as mb

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


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
