"""The wait limit of an e4m3 plan bounds its kernels' pipelines, not the kernels before them."""
from __future__ import annotations

import pytest
import torch

from sparse_moe_layer_row_gb300 import moe_block as mb
from tests import fp8_ref as F

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    mb.load()


def randn(*shape, seed=0, sigma=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda") * sigma


def test_wait_limit_counts_the_pipeline_alone():
    """A wait limit below the gate/up GEMM's time and far above any wait of a pipeline: no call
    runs into it.  One long gate/up unit per expert leaves most SMs to the down GEMM, which
    starts early there, and each of its CTAs has more weight tiles than its ring holds."""
    H, E, I, R = 16384, 16, 64, 32
    def codes(*shape, seed):
        return F.block_codes(randn(*shape, seed=seed, sigma=0.02))
    (wg, gs), (wu, us), (wd, ds) = codes(E, I, H, seed=1), codes(E, I, H, seed=2), codes(E, H, I, seed=3)
    (sg, sgs), (su, sus), (sd, sds) = codes(I, H, seed=4), codes(I, H, seed=5), codes(H, I, seed=6)
    q = mb.Fp8Experts(wg, wu, wd, gs, us, ds, sg, su, sd, sgs, sus, sds)
    router = torch.zeros(E, H, dtype=torch.bfloat16, device="cuda")
    layer = mb.MoeBlockLayer.fp8(router, q, k=1, max_rows=R, max_blocks=1)
    mb.moe_clear_device_status(layer.workspace)
    x = randn(R, H, seed=7).to(torch.bfloat16)
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    idx = (torch.arange(R, device="cuda") % E).to(torch.int32)[:, None].contiguous()
    w = torch.ones(R, 1, device="cuda")
    keep = torch.full((1, 1), -1, dtype=torch.int32, device="cuda")

    def run():
        y = torch.full((R, H), float("nan"), dtype=torch.bfloat16, device="cuda")
        layer.forward(x, off, idx, w, keep, y=y)
        return y
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(5)]
    for e in ev:
        e.record()
    layer.plan.set_forward_events(ev)
    run()
    first = run()
    torch.cuda.synchronize()
    gu_us = ev[1].elapsed_time(ev[2]) * 1e3
    layer.plan.set_forward_events(None)
    assert gu_us > 40, gu_us                 # far above what a pipeline waits for
    layer.plan.set_wait_limit(int(gu_us * 500))   # half of it, in ns
    try:
        outs = [run() for _ in range(10)]
        torch.cuda.synchronize()
        st = layer.status()
    finally:
        layer.plan.set_wait_limit(0)
    assert st["wait_timeout"] == 0 and not any(st.values()), (gu_us, st)
    assert all(torch.equal(y, first) for y in outs) and not torch.isnan(first).any()
