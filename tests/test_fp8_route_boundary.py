"""Host-side checks of the scored routing and the e4m3 calls (no GPU needed): bad
arguments are refused with a status and a message before any CUDA work."""
from __future__ import annotations

import ctypes

import pytest
import torch

from sparse_moe_layer_row_gb300 import build as cbuild
from sparse_moe_layer_row_gb300 import moe_block as mb
from tests import fp8_ref as F

P = ctypes.c_void_p
OK = P(0x100000)      # never reached: every call here is refused on the host


@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return mb.load()


def rule(**kw):
    d = dict(score=0, n_groups=8, top_groups=4, group_score=1, renormalize=1, scale=1.0)
    d.update(kw)
    return mb.moe_route_rule(*[d[n] for n, _ in mb.moe_route_rule._fields_])


def call_route(lib, r=None, logits=OK, dtype=2, ld=256, R=4, E=256, k=8, bias=None, idx=OK, w=OK, sc=None):
    r = rule() if r is None else r
    return lib.moe_route_scored(ctypes.byref(r), logits, dtype, ld, R, E, k, bias, idx, w, sc, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(logits=None), -1, "logits"), (dict(logits=P(0x100002)), -1, "logits"),
    (dict(idx=None), -1, "topk"), (dict(w=P(0x100001)), -1, "topk"), (dict(sc=P(0x100001)), -1, "output"),
    (dict(bias=P(0x100002)), -1, "select_bias"), (dict(dtype=3), -2, "dtype"), (dict(R=-1), -1, "R="),
    (dict(E=0), -2, "E="), (dict(E=1025, ld=2000), -2, "E="), (dict(k=0), -2, "k="), (dict(k=33), -2, "k="),
    (dict(ld=255), -1, "row_stride"), (dict(r=rule(score=2)), -1, "score"),
    (dict(r=rule(group_score=2)), -1, "group_score"), (dict(r=rule(n_groups=0)), -2, "n_groups"),
    (dict(r=rule(n_groups=33)), -2, "n_groups"), (dict(r=rule(n_groups=7)), -2, "n_groups"),
    (dict(r=rule(top_groups=0)), -1, "top_groups"), (dict(r=rule(top_groups=9)), -1, "top_groups"),
    (dict(E=16, k=9, ld=16), -1, "k=9"), (dict(r=rule(scale=float("nan"))), -1, "scale"),
    (dict(r=rule(scale=float("inf"))), -1, "scale")], ids=str)
def test_route_scored_refuses(lib, kw, status, word):
    assert call_route(lib, **kw) == status
    assert word in lib.moe_last_error().decode()


def test_route_scored_null_rule_and_no_rows(lib):
    assert lib.moe_route_scored(None, OK, 2, 256, 4, 256, 8, None, OK, OK, None, None) == -1
    assert call_route(lib, R=0, logits=None, idx=None, w=None) == 0
    assert lib.moe_last_error() == b""


def test_route_rule_names():
    for bad in (dict(score="argmax"), dict(group_score="mean")):
        with pytest.raises(ValueError):
            mb.RouteRule(**bad)


def call_quant(lib, x=OK, dtype=0, ld=256, R=4, K=256, codes=OK, scales=OK):
    return lib.moe_fp8_quantize(x, dtype, ld, R, K, codes, scales, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(x=None), -1, "x "), (dict(x=P(0x100001)), -1, "x "), (dict(dtype=2, x=P(0x100002)), -1, "x "),
    (dict(dtype=-1), -2, "dtype"), (dict(ld=255), -1, "row_stride"), (dict(R=-1), -1, "R="),
    (dict(K=0), -1, "K="), (dict(codes=None), -1, "codes"), (dict(scales=None), -1, "scales"),
    (dict(scales=P(0x100002)), -1, "scales")], ids=str)
def test_quantize_refuses(lib, kw, status, word):
    assert call_quant(lib, **kw) == status
    assert word in lib.moe_last_error().decode()


def test_quantize_no_rows(lib):
    assert call_quant(lib, R=0, x=None, codes=None, scales=None) == 0


def call_gemm(lib, xq=OK, xs=OK, R=4, wq=OK, ws=OK, N=256, K=256, y=OK, dtype=0, ld=256, mem=OK, nbytes=1 << 30):
    return lib.moe_fp8_gemm(xq, xs, R, wq, ws, N, K, y, dtype, ld, mem, nbytes, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(xq=None), -1, "xq"), (dict(xq=P(0x100008)), -1, "xq"), (dict(wq=P(0x100004)), -1, "wq"),
    (dict(xs=None), -1, "xs"), (dict(ws=P(0x100002)), -1, "ws"), (dict(K=100), -2, "K="),
    (dict(K=0), -1, "K="), (dict(N=0), -1, "N="), (dict(R=-1), -1, "R="), (dict(ld=255), -1, "row_stride"),
    (dict(dtype=7), -2, "dtype"), (dict(y=None), -1, "y "), (dict(y=P(0x100001)), -1, "y "),
    (dict(dtype=2, y=P(0x100002)), -1, "y "), (dict(mem=None), -3, "workspace"),
    (dict(mem=P(0x100010)), -3, "workspace"), (dict(nbytes=16), -3, "workspace")], ids=str)
def test_gemm_refuses(lib, kw, status, word):
    assert call_gemm(lib, **kw) == status
    assert word in lib.moe_last_error().decode()


def test_gemm_no_rows_and_workspace(lib):
    assert call_gemm(lib, R=0, xq=None, xs=None, wq=None, ws=None, y=None, mem=None) == 0
    assert mb.moe_fp8_gemm_workspace_bytes(1, 1, 16) >= 256
    for bad in ((-1, 1, 16), (1, 0, 16), (1, 1, 0), (1, 1, 24)):
        with pytest.raises(mb.MoeError):
            mb.moe_fp8_gemm_workspace_bytes(*bad)


def dims(**kw):
    d = dict(H=2048, E=256, k=8, I=512, Is=512, max_rows=32, max_blocks=1)
    d.update(kw)
    return mb.moe_dims(**d)


def test_plan_create_fp8_refuses(lib):
    h = P()
    names = [n for n, _ in mb.moe_fp8_weights._fields_]

    def create(d=None, router=OK, out=ctypes.byref(h), weights=True, **kw):
        v = {n: 0x100000 for n in names}
        v.update(kw)
        w = mb.moe_fp8_weights(*[v[n] for n in names])
        return lib.moe_plan_create_fp8(ctypes.byref(d or dims()), router, ctypes.byref(w) if weights else None, out)
    assert create(out=None) == -1
    assert create(weights=False) == -1 and b"NULL" in lib.moe_last_error()
    assert create(router=None) == -1 and b"w_router" in lib.moe_last_error()
    for n in names:
        for bad in (None, 0x100002):
            assert create(**{n: bad}) == -1
            assert n.encode() in lib.moe_last_error()
    for bad in (dict(H=100), dict(I=100), dict(Is=0), dict(E=0), dict(k=33)):
        assert create(d=dims(**bad)) == -2
    assert not h.value


def test_block_logits_refuses(lib):
    assert lib.moe_block_logits(None, OK, 4, OK, 1, None, OK, OK, 1 << 20, None) == -1
    assert b"plan" in lib.moe_last_error()


def test_header_struct_fields():
    """The binding's structs have the header's fields in the header's order."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    hdr = open(os.path.join(root, "include", "moe_block.h")).read()
    for cls in (mb.moe_fp8_weights, mb.moe_route_rule):
        body = re.search(r"typedef struct %s \{(.*?)\}" % cls.__name__, hdr, re.S).group(1)
        assert re.findall(r"(\w+)\s*[,;]", body) == [f for f, _ in cls._fields_]


def test_binding_refuses_cpu_and_misfit_tensors():
    z = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        mb.moe_route_scored(z, mb.RouteRule(), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2))
    with pytest.raises(ValueError):
        mb.moe_fp8_quantize(z, z, z)
    with pytest.raises(ValueError):
        mb.moe_fp8_gemm(z, z, z, z, z, z)
    with pytest.raises(TypeError):
        mb.moe_fp8_quantize([1.0], z, z)


def test_synthetic_e4m3_experts():
    """quantize_blocks_e4m3: shapes, the scale of each block, values within half a code's
    step of the weights (2^-4 of the value, or of the least normal code)."""
    from sparse_moe_layer_row_gb300 import workloads as W
    w = torch.randn(3, 200, 300)
    w[1, :128, :128] = 0.0
    q, s = W.quantize_blocks_e4m3(w)
    assert q.shape == w.shape and s.shape == (3, 2, 3) and q.dtype == torch.float8_e4m3fn
    assert s[1, 0, 0] == torch.tensor(2.0 ** -100) / 448.0
    assert s[0, 1, 2] == w[0, 128:, 256:].abs().max() / 448.0
    v = F.weight_values(q, s)
    step = s.repeat_interleave(128, -2)[..., :200, :].repeat_interleave(128, -1)[..., :300].double() * 2.0 ** -6
    assert torch.all((v - w.double()).abs() <= 2.0 ** -4 * torch.maximum(w.abs().double(), step) * (1 + 1e-6))
    T = W.make_tensors(W.TINY)
    e = W.fp8_experts(T, chunk=5)
    assert e.gate.shape == (16, 128, 256) and e.gate_scale.shape == (16, 1, 2)
    assert e.down.shape == (16, 256, 128) and e.shared_down_scale.shape == (2, 1)
    one, os_ = W.quantize_blocks_e4m3(T.w_up[7])
    assert torch.equal(e.up[7].view(torch.uint8), one.view(torch.uint8)) and torch.equal(e.up_scale[7], os_)


# ---- the references that the GPU tests compare with

def test_reference_rounding_matches_the_type():
    v = torch.linspace(-448, 448, 20001, dtype=torch.float64)
    assert torch.equal(F.e4m3_round(v), v.float().to(torch.float8_e4m3fn).double())
    q, s = F.quantize(torch.randn(5, 300))
    assert q.abs().max() == 448 and s.shape == (3, 5)


def test_reference_routing_by_hand():
    z = torch.tensor([0.0, 2.0, 1.0, 2.0, -1.0, 3.0, float("-inf"), 0.5]).numpy().astype("f8")
    ids, w, s = F.route(z, mb.RouteRule(), 3)
    assert list(ids) == [5, 1, 3] and abs(w.sum() - 1) < 1e-15
    ids, w, s = F.route(z, mb.RouteRule(n_groups=4, top_groups=1, score="sigmoid", renormalize=False), 2)
    assert list(ids) == [5, 4]
    ids, _, _ = F.route(z, mb.RouteRule(n_groups=4, top_groups=2, group_score="top2", score="sigmoid"), 2,
                        bias=torch.tensor([0, 0, 0, 0, .9, 0, 0, 0.]).numpy())
    assert list(ids) == [4, 5]
    ids, w, _ = F.route(z * 0 + float("-inf"), mb.RouteRule(), 2)
    assert list(ids) == [0, 1] and not w.any()
