"""moe_add_rmsnorm of no rows takes null buffers, as an empty tensor's are, whatever it writes
(no GPU needed)."""
from __future__ import annotations

import ctypes

import pytest

from sparse_moe_layer_row_gb300 import build as cbuild
from sparse_moe_layer_row_gb300 import moe_block as mb

P = ctypes.c_void_p
AT = P(0x100000)   # never read


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("buffers", [None, AT], ids=["null", "given"])
@pytest.mark.parametrize("residual", [None, AT], ids=["alone", "residual"])
def test_norm_of_no_rows(kind, buffers, residual):
    cbuild.build()
    lib = mb.load()
    out = buffers if kind else None
    assert lib.moe_add_rmsnorm(buffers, 0, 256, 0, 256, residual, 0, 256, residual, 256, None, 0, 1e-6, buffers, 256,
                               kind, out, out, None) == 0
    assert lib.moe_last_error() == b""


def test_norm_of_no_rows_still_checks_the_rest():
    lib = mb.load()
    for kw, word in ((dict(dtype=3), b"dtype"), (dict(H=0), b"H="), (dict(eps=0.0), b"eps"), (dict(kind=3), b"code_type"),
                     (dict(ldx=255), b"x_stride")):
        a = dict(dtype=0, ldx=256, H=256, eps=1e-6, kind=1) | kw
        assert lib.moe_add_rmsnorm(None, a["dtype"], a["ldx"], 0, a["H"], None, 0, 256, None, 256, None, 0, a["eps"],
                                   None, 256, a["kind"], None, None, None) != 0
        assert word in lib.moe_last_error()
