"""The layer for a few rows at the ends of its sizes."""
from __future__ import annotations

import pytest
import torch

from sparse_moe_layer_row_gb300 import moe_block as mb
from tests.test_gpu_token import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    mb.load()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("R", [1, 3])
def test_wide_shared_expert(R, kind):
    """A shared expert of which more tiles fall to a CTA than it asks for ahead."""
    c = Case(kind, R, H=2048, E=8, k=2, I=64, Is=16384, seed=90 + R, sigma=0.02)
    y, y32, idx, wt = c.routed()
    c.check(y, y32, c.reference(idx, wt))
    g = c.given(idx, wt)
    assert torch.equal(g[1], y32)
    c.status_clean()
