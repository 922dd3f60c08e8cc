"""The e4m3 operators at the ends of what they accept."""
from __future__ import annotations

import pytest
import torch

from sparse_moe_layer_row_gb300 import moe_block as mb
from tests import fp8_ref as F

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    mb.load()


def randn(*shape, seed=0, sigma=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda") * sigma


def test_gemm_outputs_of_2_31_bytes_a_row():
    """fp32 rows of 2^29 outputs: byte counts within a row pass 31 bits.  33 rows take the
    128-row tiles.  71 GB of outputs, of which both ends and the middle are compared."""
    R, N, K, per = 33, 1 << 29, 16, 1 << 14
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB")
    q, s = F.block_codes(randn(per, K, seed=1, sigma=0.02))
    wq = q.view(torch.uint8).repeat(N // per, 1).view(E4M3)
    ws = s.repeat(N // per, 1)
    xq = torch.empty(R, K, dtype=torch.uint8, device="cuda").view(E4M3)
    xs = torch.empty(1, R, device="cuda")
    mb.moe_fp8_quantize(randn(R, K, seed=2), xq, xs)
    mem = torch.zeros(mb.moe_fp8_gemm_workspace_bytes(R, N, K), dtype=torch.uint8, device="cuda")
    y = torch.empty(R, N, device="cuda")
    ref, bound = F.gemm(xq, xs, q, s)
    tol = bound + (ref.abs() + bound) * F.HALF[torch.float32] + 1e-30
    at = [0, per, N // 2, N - per]
    for a in at:
        y[:, a:a + per] = float("nan")
    mb.moe_fp8_gemm(xq, xs, wq, ws, y, mem)
    torch.cuda.synchronize()
    bad = {a: int((~((y[:, a:a + per].double() - ref).abs() <= tol)).sum()) for a in at}
    status = mb.moe_read_device_status(mem)
    del y, wq, ws
    torch.cuda.empty_cache()
    assert not any(bad.values()), bad
    assert not any(status.values()), status
