"""The e4m3 block-scaled operators against plain 64-bit references (tests/fp8_ref.py):
quantising rows, the dense product, and the expert FFN of an e4m3 plan."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from sparse_moe_layer_row_gb300 import moe_block as mb, workloads as W
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


# ------------------------------------------------------------------------- quantise

def quantize(x, stream=None):
    R, K = x.shape
    q = torch.zeros(R, K, dtype=torch.uint8, device="cuda").view(E4M3)
    s = torch.full((-(-K // 128), R), float("nan"), device="cuda")
    mb.moe_fp8_quantize(x, q, s, stream=stream)
    torch.cuda.synchronize()
    return q, s


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("R,K", [(1, 128), (1, 1), (3, 7), (32, 2048), (5, 1000), (70, 136), (257, 640), (2, 4104)])
def test_quantize(R, K, dtype):
    x = (randn(R, K, seed=R + K) * torch.exp(2 * randn(R, 1, seed=7))).to(dtype)
    q, s = quantize(x)
    rq, rs = F.quantize(x)
    assert torch.equal(s.double(), rs)
    if dtype == torch.float32:
        # 7/8 x may round once more: codes may differ where 448 x / a is that near a midpoint
        p = F.pad_blocks(x.double())
        v = (448.0 * p / p.abs().amax(-1, keepdim=True).clamp_min(2.0 ** -100)).view(R, -1)[:, :K]
        gap, _ = F.e4m3_midpoint_gap(v)
        assert torch.all((q.double() == rq) | (gap <= 2 * F.STEP * v.abs()))
    else:
        assert torch.equal(q.double(), rq)


def test_quantize_fp32_quotient_rule():
    """fp32 values: the codes of (7/8 v) / (a / 512), each operation rounded to fp32, also
    where that is a middle of two codes that 448 v / a only comes close to."""
    x = randn(4096, 2048, seed=11)
    q, _ = quantize(x)
    p = x.view(4096, 16, 128)
    v = p * 0.875 / (p.abs().amax(-1, keepdim=True) * 2.0 ** -9)
    assert torch.equal(q.view(torch.uint8), v.to(E4M3).view(4096, 2048).view(torch.uint8))


def test_quantize_ties_zeros_tiny_and_huge():
    """Values exactly between two codes go to the even one; blocks of zeros, subnormals and
    the largest finite values stay finite."""
    t = torch.tensor(F.E4M3, dtype=torch.float64)
    mids = ((t[1:] + t[:-1]) / 2).float()
    x = torch.zeros(6, 384, device="cuda")
    x[0, 0] = 448.0
    x[0, 1:127] = mids.cuda()
    x[1, 128] = -448.0 * 2 ** 20
    x[1, 129:255] = -(mids * 2.0 ** 20).cuda()
    x[2] = 1e-38
    x[3, 5] = torch.finfo(torch.float32).max
    x[3, 6] = -torch.finfo(torch.float32).max / 3
    x[4, 383] = -2.0 ** -120
    for dt in (torch.float32, torch.bfloat16):
        xx = x.to(dt)
        if dt == torch.bfloat16:
            xx = xx.clamp(-3e38, 3e38)
        q, s = quantize(xx)
        rq, rs = F.quantize(xx)
        assert torch.equal(q.double(), rq) and torch.equal(s.double(), rs)
        assert torch.isfinite(s).all() and torch.isfinite(q.float()).all()


def test_quantize_nan_and_infinity_poison_their_block_only():
    x = randn(3, 384, seed=1)
    x[0, 130] = float("nan")
    x[1, 5] = float("inf")
    x[1, 6] = float("nan")
    x[2, 300] = float("-inf")
    q, s = quantize(x)
    rq, rs = F.quantize(torch.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0))
    bad = torch.zeros(3, 3, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[1, 0] = bad[2, 2] = True
    assert torch.equal(s.t()[~bad].double(), rs.t()[~bad])
    wide = bad.repeat_interleave(128, 1)
    assert torch.equal(q.double()[~wide], rq[~wide])
    assert torch.isnan(s[1, 0]) and torch.isnan(s[0, 1]) and torch.isinf(s[2, 2])
    assert torch.isnan(F.row_values(q, s)[wide]).all()


def test_quantize_strided_rows_and_stream():
    wide = randn(40, 700, seed=2).to(torch.bfloat16)
    for c0, K in ((0, 512), (8, 512), (3, 512), (1, 130)):
        x = wide[:, c0:c0 + K]
        q, s = quantize(x)
        q2, s2 = quantize(x.contiguous())
        assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    q3, s3 = quantize(wide[:, 1:131], stream=st)
    assert torch.equal(q3.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s3, s2)


# ---------------------------------------------------------------------------- dense

def gemm(xq, xs, wq, ws, dtype=torch.bfloat16, y=None):
    R, K = xq.shape
    N = wq.shape[0]
    mem = torch.zeros(mb.moe_fp8_gemm_workspace_bytes(R, N, K), dtype=torch.uint8, device="cuda")
    if y is None:
        y = torch.full((R, N), float("nan"), dtype=dtype, device="cuda")
    mb.moe_fp8_gemm(xq, xs, wq, ws, y, mem)
    torch.cuda.synchronize()
    st = mb.moe_read_device_status(mem)
    assert not any(st.values()), st
    return y


def operands(R, N, K, seed=0, sigma=0.02):
    xq, xs = quantize(randn(R, K, seed=seed) * torch.exp(randn(R, 1, seed=seed + 1)))
    wq, ws = F.block_codes(randn(N, K, seed=seed + 2, sigma=sigma))
    return xq, xs, wq, ws


def assert_gemm(y, ref, bound):
    tol = bound + (ref.abs() + bound) * F.HALF[y.dtype] + 1e-30
    err = (y.double() - ref).abs()
    assert torch.all(err <= tol), (float((err / tol).max()), int((err > tol).sum()))


SIZES = [(1, 1, 16), (1, 2048, 2048), (1, 1000, 1104), (2, 129, 144), (7, 256, 128), (8, 64, 4096),
         (16, 520, 256), (31, 511, 1040), (77, 1000, 1104), (128, 256, 512), (129, 257, 272),
         (300, 640, 2048), (1000, 130, 384)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("R,N,K", SIZES)
def test_gemm(R, N, K, dtype):
    ops = operands(R, N, K, seed=R + N)
    ref, bound = F.gemm(*ops)
    assert_gemm(gemm(*ops, dtype=dtype), ref, bound)


@pytest.mark.parametrize("R", range(1, 40, 3))
def test_gemm_row_counts(R):
    ops = operands(R, 384, 640, seed=R)
    ref, bound = F.gemm(*ops)
    assert_gemm(gemm(*ops, dtype=torch.float32), ref, bound)


def test_gemm_few_outputs_of_very_many_rows():
    """More row tiles than a grid has in y, with too few outputs to fill a tile."""
    ops = operands(65535 * 32 + 5, 16, 16, seed=8)
    ref, bound = F.gemm(*ops)
    assert_gemm(gemm(*ops, dtype=torch.float32), ref, bound)


@pytest.mark.parametrize("R", [1, 5, 50, 200])
def test_gemm_large_codes_and_unlike_scales(R):
    """Codes over the whole range and scales orders of magnitude apart."""
    N, K = 200, 400
    g = torch.Generator(device="cuda").manual_seed(3)
    t = torch.tensor(np.concatenate([F.E4M3, -F.E4M3]), device="cuda", dtype=torch.float32)
    xq = t[torch.randint(0, len(t), (R, K), generator=g, device="cuda")].to(E4M3)
    wq = t[torch.randint(0, len(t), (N, K), generator=g, device="cuda")].to(E4M3)
    xs = torch.exp(8 * torch.randn(4, R, generator=g, device="cuda"))
    ws = torch.exp(8 * torch.randn(2, 4, generator=g, device="cuda"))
    ref, bound = F.gemm(xq, xs, wq, ws)
    assert_gemm(gemm(xq, xs, wq, ws, dtype=torch.float32), ref, bound)


@pytest.mark.parametrize("R", [1, 6, 140])
def test_gemm_strided_output_and_guard(R):
    """Rows of a wider buffer, at aligned and odd offsets: nothing beside them is written."""
    ops = operands(R, 300, 256, seed=4)
    ref, bound = F.gemm(*ops)
    for dt in (torch.bfloat16, torch.float32):
        for c0 in (0, 8, 1):
            buf = torch.full((R + 2, 333), 7.0, dtype=dt, device="cuda")
            y = buf[1:-1, c0:c0 + 300]
            gemm(*ops, y=y)
            assert_gemm(y, ref, bound)
            mask = torch.ones_like(buf, dtype=torch.bool)
            mask[1:-1, c0:c0 + 300] = False
            assert torch.all(buf[mask] == 7.0)


@pytest.mark.parametrize("R", [2, 9, 130])
def test_gemm_nan_rows_stay_apart(R):
    """A NaN or infinite row of x poisons its own row of y and no other."""
    xq, xs, wq, ws = operands(R, 260, 400, seed=5)
    clean = gemm(xq, xs, wq, ws, dtype=torch.float32)
    xs2 = xs.clone()
    xs2[1, R - 1] = float("nan")
    y = gemm(xq, xs2, wq, ws, dtype=torch.float32)
    assert torch.isnan(y[R - 1]).all() and torch.equal(y[:R - 1], clean[:R - 1])
    codes = xq.clone()
    codes.view(torch.uint8)[0, 399] = 0x7F
    y = gemm(codes, xs, wq, ws, dtype=torch.float32)
    assert torch.isnan(y[0]).all() and torch.equal(y[1:], clean[1:])


def test_gemm_no_rows_and_repeats():
    wq, ws = F.block_codes(randn(64, 128, seed=1))
    empty = torch.empty(0, 128, dtype=torch.uint8, device="cuda").view(E4M3)
    assert gemm(empty, torch.empty(1, 0, device="cuda"), wq, ws).shape == (0, 64)
    for R in (3, 300):
        ops = operands(R, 700, 512, seed=6)
        a, b = gemm(*ops), gemm(*ops)
        assert torch.equal(a, b)


# -------------------------------------------------------------------------- experts

class Ffn:
    """An e4m3 layer with seeded weights, its routing, and the 64-bit reference."""

    def __init__(self, R, H=256, E=16, k=4, I=128, Is=128, block=32, seed=0, sigma=0.05, drop=0.1):
        self.R, self.H, self.E, self.k = R, H, E, k
        g = torch.Generator(device="cuda").manual_seed(seed + 100)

        def codes(*shape):
            return F.block_codes(torch.randn(*shape, generator=g, device="cuda") * sigma)
        (wg, gs), (wu, us), (wd, ds) = codes(E, I, H), codes(E, I, H), codes(E, H, I)
        (sg, sgs), (su, sus), (sd, sds) = codes(Is, H), codes(Is, H), codes(H, Is)
        self.q = mb.Fp8Experts(wg, wu, wd, gs, us, ds, sg, su, sd, sgs, sus, sds)
        self.router = torch.randn(E, H, generator=g, device="cuda").to(torch.bfloat16) * 0.05
        self.x = torch.randn(R, H, generator=g, device="cuda").to(torch.bfloat16)
        z = torch.randn(R, E, generator=g, device="cuda")
        self.idx = z.argsort(dim=1, descending=True)[:, :k].to(torch.int32).contiguous()
        self.w = torch.softmax(torch.randn(R, k, generator=g, device="cuda"), dim=1)
        nb = max(1, -(-R // block))
        self.off = (torch.arange(nb + 1, device="cuda") * block).clamp_max(R).to(torch.int32)
        self.kept = torch.rand(nb, E, generator=g, device="cuda") >= drop
        if nb > 2:
            self.kept[1] = False          # a block whose rows keep the shared expert alone
        self.block_of = torch.arange(R, device="cuda") // block
        self.keep = pack_bits(self.kept)
        self.layer = mb.MoeBlockLayer.fp8(self.router, self.q, k=k, max_rows=max(R, 1), max_blocks=nb)
        mb.moe_clear_device_status(self.layer.workspace)

    def run(self, live=None, y=None, y32=None):
        y = torch.full((self.R, self.H), float("nan"), dtype=torch.bfloat16, device="cuda") if y is None else y
        y32 = torch.full((self.R, self.H), float("nan"), device="cuda") if y32 is None else y32
        self.layer.forward(self.x, self.off, self.idx, self.w, self.keep, y=y, y_f32=y32, live=live)
        torch.cuda.synchronize()
        return y, y32

    def reference(self):
        """(y, bound on the error of the fp32 sum)."""
        q = self.q
        x = F.row_values(*F.quantize(self.x))
        y, b = F.swiglu(x, F.weight_values(q.shared_gate, q.shared_gate_scale),
                        F.weight_values(q.shared_up, q.shared_up_scale),
                        F.weight_values(q.shared_down, q.shared_down_scale))
        bound = b + (y.abs() + b) * 2.0 ** -11 + 2.0 ** -25       # staged in fp16 (its subnormal step)
        mag = y.abs()
        for e in range(self.E):
            hit = (self.idx == e) & self.kept[self.block_of, e][:, None]
            r, j = torch.nonzero(hit, as_tuple=True)
            if not len(r):
                continue
            o, b = F.swiglu(x[r], F.weight_values(q.gate[e], q.gate_scale[e]),
                            F.weight_values(q.up[e], q.up_scale[e]),
                            F.weight_values(q.down[e], q.down_scale[e]))
            w = self.w[r, j].double()[:, None]
            # index_add: a row may name an expert twice
            y.index_add_(0, r, w * o)
            mag.index_add_(0, r, (w * o).abs())
            bound.index_add_(0, r, w * (b + (o.abs() + b) * (2.0 ** -11 + 2.0 ** -23)) + 2.0 ** -25)
        return y, bound + (mag + bound) * (self.k + 1) * 2.0 ** -24

    def check(self, y, y32, rows=slice(None)):
        ref, bound = self.reference()
        for got in (y32, y):
            tol = bound + (ref.abs() + bound) * F.HALF[got.dtype]
            err = (got.double() - ref).abs()
            frac = float((err / tol)[rows].max()) if got[rows].numel() else 0.0
            assert torch.all((err <= tol)[rows]), frac
        st = self.layer.status()
        assert not any(st.values()), st


def pack_bits(kept):
    nb, E = kept.shape
    p = torch.nn.functional.pad(kept, (0, -E % 32)).view(nb, -1, 32).long()
    bits = (p << torch.arange(32, device=kept.device)).sum(-1)
    return torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).to(torch.int32).contiguous()


SHAPES = [dict(), dict(I=64, Is=192), dict(I=320, Is=64, H=512, E=24, k=3), dict(I=192, Is=320, E=40, k=8, block=8)]


@pytest.mark.parametrize("R", [1, 2, 7, 8, 9, 31, 32, 33, 130, 300])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_experts(shape, R):
    f = Ffn(R, seed=R, **shape)
    f.check(*f.run())


def test_experts_rows_past_a_tile():
    """Few experts and many rows: several 128-row units per expert, cut short."""
    f = Ffn(700, E=3, k=2, block=50, seed=8)
    f.check(*f.run())


def test_experts_full_shape():
    f = Ffn(40, H=2048, E=256, k=8, I=512, Is=512, seed=9, sigma=0.02)
    f.check(*f.run())


@pytest.mark.parametrize("R", [1, 3])
def test_experts_full_shape_few_rows(R):
    f = Ffn(R, H=2048, E=256, k=8, I=512, Is=512, seed=R, sigma=0.02, drop=0.0)
    f.check(*f.run())


@pytest.mark.parametrize("R", [1, 6, 40, 300])
def test_experts_one_expert_takes_all(R):
    """Every row on the same experts: as many pairs per expert as rows, the others untouched."""
    f = Ffn(R, E=24, k=2, seed=20 + R, drop=0.0)
    f.idx[:, 0] = 5
    f.idx[:, 1] = 23
    f.check(*f.run())


@pytest.mark.parametrize("R", [1, 2, 8, 40, 300])
def test_experts_large_outputs(R):
    """Outputs beyond fp16's range: the staged exponent."""
    f = Ffn(R, seed=10, sigma=3.0)
    y, y32 = f.run()
    assert float(y32.abs().max()) > 65504
    f.check(y, y32)


@pytest.mark.parametrize("R", [4, 32, 150])
def test_experts_live_rows(R):
    f = Ffn(R, seed=11)
    full = f.run()
    live = (torch.rand(R, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) < 0.4)
    live[0] = True
    y = torch.full((R, f.H), 3.0, dtype=torch.bfloat16, device="cuda")
    y32 = torch.full((R, f.H), 3.0, device="cuda")
    f.run(live=live.to(torch.uint8), y=y, y32=y32)
    assert torch.equal(y[live], full[0][live]) and torch.equal(y32[live], full[1][live])
    assert torch.all(y[~live] == 3.0) and torch.all(y32[~live] == 3.0)


@pytest.mark.parametrize("R", [5, 32, 200])
def test_experts_repeat_and_row_independence(R):
    """Same call, same bits; a row's output does not depend on the rows beside it."""
    f = Ffn(R, seed=12)
    a, b = f.run(), f.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    f.x[R // 2] = float("nan")
    c = f.run()
    mask = torch.ones(R, dtype=torch.bool, device="cuda")
    mask[R // 2] = False
    assert torch.equal(a[1][mask], c[1][mask]) and torch.isnan(c[1][R // 2]).all()
    assert f.layer.status()["nonfinite_output"] > 0


def test_experts_bad_ids_are_skipped():
    f = Ffn(40, seed=13)
    f.idx[3, 1] = -5
    f.idx[7, 0] = 1 << 20
    f.idx[9, 2] = f.idx[9, 0]            # named twice: the first slot counts
    y, y32 = f.run()
    ok = f.idx.clone()
    ref = Ffn(40, seed=13)
    ref.idx.copy_(ok)
    ref.idx[3, 1] = ref.idx[3, 0]        # the reference drops them by weight
    w = ref.w
    w[3, 1] = 0.0
    w[7, 0] = 0.0
    ref.idx[7, 0] = ref.idx[7, 1]
    w[9, 2] = 0.0
    rr, bound = ref.reference()
    assert torch.all((y32.double() - rr).abs() <= bound + (rr.abs() + bound) * 2.0 ** -24)


@pytest.mark.parametrize("R", [1, 32, 300])
def test_pass_equals_the_three_calls(R):
    f = Ffn(R, H=512, E=32, k=4, seed=14)
    L = f.layer
    idx, w = L.route(f.x, f.off)
    keep, core, wr, empty = L.coreset(f.off, idx, w, 0.9)
    y = L.forward(f.x, f.off, idx, wr, keep).clone()
    z = L(f.x, f.off, 0.9)
    torch.cuda.synchronize()
    assert torch.equal(y, z) and not torch.isnan(y).any()


def test_scored_routing_through_the_layer():
    """route_scored -> coreset over its scores -> e4m3 experts, as a user runs them, also
    captured as a graph."""
    f = Ffn(64, H=512, E=32, k=4, seed=15)
    L = f.layer
    rule = mb.RouteRule(score="sigmoid", n_groups=4, top_groups=2, group_score="top2", scale=2.5)
    bias = randn(32, seed=3, sigma=0.05)
    y = torch.empty(64, 512, dtype=torch.bfloat16, device="cuda")

    def step():
        idx, w, s = L.route_scored(f.x, f.off, rule, select_bias=bias)
        keep, core, wr, empty = L.coreset(f.off, idx, w, 1.0, mass=s)
        L.forward(f.x, f.off, idx, wr, keep, y=y)
        return idx, wr, keep
    idx, wr, keep = step()
    torch.cuda.synchronize()
    first = y.clone()
    f.idx, f.w = idx.clone(), wr.clone()
    f.kept[:] = True
    ref, bound = f.reference()
    assert torch.all((first.double() - ref).abs() <= bound + (ref.abs() + bound) * 2.0 ** -8)
    y.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, first)


@pytest.mark.parametrize("R", [32, 300])
def test_wait_limit_aborts_and_recovers(R):
    """Every pipeline wait gives up after 1 ns: the call returns, counts the timeouts, and
    the next call with the built-in limit is right."""
    f = Ffn(R, seed=16)
    before = f.run()
    f.layer.plan.set_wait_limit(1)
    try:
        f.run()
        st = f.layer.status()
    finally:
        f.layer.plan.set_wait_limit(0)
    assert st["wait_timeout"] > 0
    mb.moe_clear_device_status(f.layer.workspace)
    after = f.run()
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
    assert not any(f.layer.status().values())


@pytest.mark.parametrize("args", [["--tiny"], ["--tiny", "--rows", "1"], ["--rows", "40"]], ids=str)
def test_example(args):
    """The example layer: its e4m3 experts stay near the bf16 ones.  A rounding to e4m3 is off
    by up to 2^-4 of a value, its mean square by (2^-4)^2 / 3; x, h and the three weights are
    rounded, so that independent errors add up to sqrt(5 / 3) 2^-4 = 0.08 of the norm at most."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "scored_fp8_layer.py")
    spec = importlib.util.spec_from_file_location("scored_fp8_layer", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    assert 0 < ex.main(args + ["--passes", "2"]) < 0.08
