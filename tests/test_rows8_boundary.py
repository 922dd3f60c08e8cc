"""Host-side checks of the residual norm and the int8 calls (no GPU needed): bad arguments
are refused with a status and a message before any CUDA work."""
from __future__ import annotations

import ctypes

import pytest
import torch

from sparse_moe_layer_row_gb300 import build as cbuild
from sparse_moe_layer_row_gb300 import moe_block as mb

P = ctypes.c_void_p
OK, OK2, OK3 = P(0x100000), P(0x200000), P(0x300000)   # never reached: every call is refused on the host


@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return mb.load()


def norm(lib, x=OK, dtype=0, ldx=256, R=4, H=256, res=OK2, rt=0, ldr=256, total=OK2, ldt=256, w=OK, wt=0,
         eps=1e-6, y=OK3, ldy=256, kind=0, codes=None, scales=None):
    return lib.moe_add_rmsnorm(x, dtype, ldx, R, H, res, rt, ldr, total, ldt, w, wt, eps, y, ldy, kind, codes,
                               scales, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(x=None), -1, "x "), (dict(x=P(0x100001)), -1, "x "), (dict(dtype=3), -2, "dtype"),
    (dict(R=-1), -1, "R="), (dict(H=0), -1, "H="), (dict(ldx=255), -1, "x_stride"),
    (dict(ldr=255), -1, "residual_stride"), (dict(ldt=255), -1, "total_stride"), (dict(ldy=255), -1, "y_stride"),
    (dict(rt=1), -2, "residual_dtype"), (dict(rt=7), -2, "residual_dtype"), (dict(wt=1), -2, "weight_dtype"),
    (dict(dtype=2, rt=0, wt=2), -2, "residual_dtype"), (dict(res=P(0x200001)), -1, "residual"),
    (dict(rt=2, res=P(0x200002)), -1, "residual"), (dict(rt=2, total=P(0x200002)), -1, "total"),
    (dict(wt=2, w=P(0x100002)), -1, "weight"), (dict(eps=0.0), -1, "eps"), (dict(eps=float("nan")), -1, "eps"),
    (dict(eps=-1e-6), -1, "eps"), (dict(eps=float("inf")), -1, "eps"), (dict(res=None), -1, "total without"),
    (dict(y=None), -1, "neither"), (dict(kind=3), -2, "code_type"), (dict(kind=1), -1, "codes"),
    (dict(kind=0, codes=OK), -1, "codes"), (dict(kind=2, codes=OK), -1, "codes"),
    (dict(kind=2, scales=OK), -1, "codes"), (dict(kind=1, codes=OK, scales=P(0x100002)), -1, "scales"),
    (dict(y=P(0x300001)), -1, "y "), (dict(y=OK2), -1, "same"), (dict(ldt=264), -1, "residual's place"),
    (dict(total=OK, ldt=264), -1, "x's place"), (dict(total=OK, rt=2), -1, "x's place"),
    (dict(y=OK, ldy=264), -1, "x's place")], ids=str)
def test_norm_refuses(lib, kw, status, word):
    assert norm(lib, **kw) == status
    assert word in lib.moe_last_error().decode()


def test_norm_no_rows(lib):
    assert norm(lib, R=0, x=None, y=None) == 0
    assert lib.moe_last_error() == b""


def quant(lib, x=OK, dtype=0, ld=256, R=4, K=256, codes=OK, scales=OK):
    return lib.moe_i8_quantize(x, dtype, ld, R, K, codes, scales, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(x=None), -1, "x "), (dict(x=P(0x100001)), -1, "x "), (dict(dtype=2, x=P(0x100002)), -1, "x "),
    (dict(dtype=-1), -2, "dtype"), (dict(ld=255), -1, "row_stride"), (dict(R=-1), -1, "R="),
    (dict(K=0), -1, "K="), (dict(codes=None), -1, "codes"), (dict(scales=None), -1, "scales"),
    (dict(scales=P(0x100002)), -1, "scales")], ids=str)
def test_quantize_refuses(lib, kw, status, word):
    assert quant(lib, **kw) == status
    assert word in lib.moe_last_error().decode()


def gemm(lib, xq=OK, xs=OK, R=4, wq=OK, ws=OK, N=256, K=256, y=OK, dtype=0, ld=256, mem=OK, nbytes=1 << 40):
    return lib.moe_i8_gemm(xq, xs, R, wq, ws, N, K, y, dtype, ld, mem, nbytes, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(xq=None), -1, "xq"), (dict(xq=P(0x100008)), -1, "xq"), (dict(wq=P(0x100004)), -1, "wq"),
    (dict(xs=None), -1, "xs"), (dict(ws=P(0x100002)), -1, "ws"), (dict(K=100), -2, "K="),
    (dict(K=1 << 17), -2, "K="), (dict(K=0), -1, "K="), (dict(N=0), -1, "N="), (dict(R=-1), -1, "R="),
    (dict(ld=255), -1, "row_stride"), (dict(dtype=7), -2, "dtype"), (dict(y=None), -1, "y "),
    (dict(y=P(0x100001)), -1, "y "), (dict(dtype=2, y=P(0x100002)), -1, "y "), (dict(mem=None), -3, "workspace"),
    (dict(mem=P(0x100010)), -3, "workspace"), (dict(nbytes=16), -3, "workspace")], ids=str)
def test_gemm_refuses(lib, kw, status, word):
    assert gemm(lib, **kw) == status
    assert word in lib.moe_last_error().decode()


def test_no_rows_and_workspace(lib):
    assert quant(lib, R=0, x=None, codes=None, scales=None) == 0
    assert gemm(lib, R=0, xq=None, xs=None, wq=None, ws=None, y=None, mem=None) == 0
    assert mb.moe_i8_gemm_workspace_bytes(1, 1, 16) >= 256
    for bad in ((-1, 1, 16), (1, 0, 16), (1, 1, 0), (1, 1, 24), (1, 1, 1 << 17)):
        with pytest.raises(mb.MoeError):
            mb.moe_i8_gemm_workspace_bytes(*bad)


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 256)
    for call in (lambda: mb.moe_add_rmsnorm(x, None, 1e-6, y=x), lambda: mb.moe_i8_quantize(x, x, x),
                 lambda: mb.moe_i8_gemm(x, x, x, x, x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_token_calls_refuse_a_null_plan(lib):
    assert lib.moe_token_pass(None, OK, 1, None, OK, OK, OK2, None, OK3, 1 << 30, None) == -1
    assert b"plan" in lib.moe_last_error()
    assert lib.moe_token_forward(None, OK, 1, OK, OK, OK2, None, OK3, 1 << 30, None) == -1
    assert b"plan" in lib.moe_last_error()
