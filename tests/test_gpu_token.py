"""moe_token_pass and moe_token_forward: the whole layer for a few rows in one kernel, against
plain 64-bit references.

Bounds (fp8_ref's terms): a sum over K is off by at most sum_factor(K) of its addends'
magnitudes; silu by 2^-21 + |g| 2^-23 of itself (fast exponential and quotient) and
1.1 times the error of g; bf16 keeps a routed h to 2^-8 of itself, two bf16 parts the shared
expert's to 2^-16; the sum over experts adds a rounding of 2^-24 per addend.
"""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

from sparse_moe_layer_row_gb300 import moe_block as mb, workloads as W
from tests import fp8_ref as F

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    mb.load()


def randn(*shape, seed=0, sigma=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda") * sigma


class Case:
    def __init__(self, kind, R, H=256, E=16, k=4, I=128, Is=192, seed=0, sigma=0.05, max_rows=None):
        self.kind, self.R, self.H, self.E, self.k, self.I, self.Is = kind, R, H, E, k, I, Is
        shapes = [(E, I, H), (E, I, H), (E, H, I), (Is, H), (Is, H), (H, Is)]
        ws = [randn(*s, seed=seed + i, sigma=sigma) for i, s in enumerate(shapes)]
        self.router = randn(E, H, seed=seed + 6, sigma=0.05).to(BF)
        rows = max_rows or max(R, 1)
        if kind == "e4m3":
            qs = [F.block_codes(w) for w in ws]
            self.w = [F.weight_values(q, s) for q, s in qs]
            q = mb.Fp8Experts(*[t[0] for t in qs[:3]], *[t[1] for t in qs[:3]], *[t[0] for t in qs[3:]], *[t[1] for t in qs[3:]])
            self.raw = [t[0] for t in qs]
            self.layer = mb.MoeBlockLayer.fp8(self.router, q, k=k, max_rows=rows, max_blocks=1)
        else:
            self.raw = [w.to(BF) for w in ws]
            self.w = [w.double() for w in self.raw]
            self.layer = mb.MoeBlockLayer(self.router, *self.raw, k=k, max_rows=rows, max_blocks=1)
        self.x = randn(R, H, seed=seed + 7).to(BF)
        g = torch.Generator(device="cuda").manual_seed(seed + 8)
        self.idx = torch.rand(R, E, generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
        self.wt = torch.softmax(torch.randn(R, k, generator=g, device="cuda"), 1)

    def ffn(self, x, wg, wu, wd, h_step=2.0 ** -8):
        """(o, bound) of rows x in 64 bits."""
        if self.kind == "e4m3":
            return F.swiglu(x, wg, wu, wd)
        f = F.sum_factor(self.H)
        g, u = x @ wg.t(), x @ wu.t()
        dg, du = (x.abs() @ wg.abs().t()) * f, (x.abs() @ wu.abs().t()) * f
        silu = g * torch.sigmoid(g)
        h = silu * u
        dh = 1.1 * dg * (u.abs() + du) + silu.abs() * du + h.abs() * (g.abs() * 2.0 ** -23 + 2.0 ** -21 + h_step)
        return h @ wd.t(), dh @ wd.abs().t() + (h.abs() @ wd.abs().t()) * 2 * F.sum_factor(self.I + self.Is)

    def reference(self, idx=None, wt=None, x=None):
        idx, wt = self.idx if idx is None else idx, self.wt if wt is None else wt
        x = self.x if x is None else x
        xv = F.row_values(*F.quantize(x)) if self.kind == "e4m3" else x.double()
        y, bound = self.ffn(xv, *self.w[3:], h_step=2.0 ** -16)
        mag = y.abs()
        for e in idx.unique().tolist():
            if not 0 <= e < self.E:
                continue
            m = ((idx == e) * wt.double()).sum(1)
            r = torch.nonzero((idx == e).any(1))[:, 0]
            o, b = self.ffn(xv[r], *[w[e] for w in self.w[:3]])
            y[r] += m[r, None] * o
            bound[r] += m[r, None].abs() * (b + o.abs() * F.STEP)
            mag[r] += m[r, None].abs() * o.abs()
        return y, bound + mag * (self.k + 20) * 2.0 ** -24

    def outputs(self):
        return (torch.full((self.R, self.H), float("nan"), dtype=BF, device="cuda"),
                torch.full((self.R, self.H), float("nan"), device="cuda"))

    def given(self, idx=None, wt=None, x=None, **kw):
        y, y32 = self.outputs()
        self.layer.token_forward(self.x if x is None else x, self.idx if idx is None else idx,
                                 self.wt if wt is None else wt, y=y, y_f32=y32, **kw)
        return y, y32

    def routed(self, bias=None, **kw):
        y, y32 = self.outputs()
        idx = torch.full((self.R, self.k), -7, dtype=torch.int32, device="cuda")
        wt = torch.full((self.R, self.k), float("nan"), device="cuda")
        self.layer.token_pass(self.x, bias=bias, topk_idx=idx, topk_w=wt, y=y, y_f32=y32, **kw)
        return y, y32, idx, wt

    def check(self, y, y32, ref):
        want, bound = ref
        assert torch.all((y32.double() - want).abs() <= bound), float(((y32.double() - want).abs() / bound).max())
        assert torch.equal(y, y32.to(BF))

    def status_clean(self):
        st = self.layer.status()
        assert not any(st.values()), st


SHAPES = [dict(), dict(H=512, E=24, k=3, I=192, Is=64), dict(H=1280, E=64, k=6, I=320, Is=640),
          dict(H=768, E=300, k=8, I=64, Is=64), dict(H=256, E=32, k=32, I=512, Is=1024), dict(H=2560, E=6, k=2, I=4096, Is=2112), dict(H=256, E=1024, k=32, I=64, Is=128), dict(H=256, E=1, k=1, I=64, Is=64), dict(H=256, E=31, k=7, I=128, Is=64)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_given_routing(shape, kind):
    for R in (1, 2, 5, 8):
        c = Case(kind, R, seed=R, **shape)
        mb.moe_clear_device_status(c.layer.workspace)
        y, y32 = c.given()
        torch.cuda.synchronize()
        c.check(y, y32, c.reference())
        c.status_clean()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_whole_pass(shape, kind):
    """ids and weights are moe_block_route's bit for bit, with and without a bias."""
    for R in (1, 3, 8):
        c = Case(kind, R, seed=10 + R, **shape)
        mb.moe_clear_device_status(c.layer.workspace)
        off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
        for bias in (None, randn(c.E, seed=3)):
            y, y32, idx, wt = c.routed(bias)
            ri, rw = c.layer.route(c.x, off, None if bias is None else bias[None])
            torch.cuda.synchronize()
            assert torch.equal(idx, ri) and torch.equal(wt, rw)
            c.check(y, y32, c.reference(idx, wt))
            g = c.given(idx, wt)
            assert torch.equal(g[0], y) and torch.equal(g[1], y32)
        c.status_clean()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("R", [1, 8])
def test_full_shape(R, kind):
    c = Case(kind, R, H=2048, E=256, k=8, I=512, Is=512, seed=30 + R, sigma=0.02)
    y, y32, idx, wt = c.routed()
    c.check(y, y32, c.reference(idx, wt))
    # the same layer through the calls for any number of rows
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    z = c.layer(c.x, off, 1.0)
    assert torch.all((y.float() - z.float()).abs() <= 2.0 ** -6 * z.float().abs() + 2e-3)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_widest_row(kind):
    c = Case(kind, 8, H=8192, E=8, k=2, I=64, Is=64, seed=40, sigma=0.01)
    y, y32, idx, wt = c.routed()
    c.check(y, y32, c.reference(idx, wt))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_one_expert_for_all_and_many_experts(kind):
    c = Case(kind, 8, E=64, k=2, seed=50)
    c.idx[:, 0], c.idx[:, 1] = 5, 63
    c.check(*c.given(), c.reference())
    c = Case(kind, 8, E=64, k=8, seed=51)
    c.idx.copy_(torch.arange(64, device="cuda").view(8, 8))
    c.check(*c.given(), c.reference())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_ids_twice_and_out_of_range_and_odd_weights(kind):
    c = Case(kind, 6, E=24, k=4, seed=52)
    mb.moe_clear_device_status(c.layer.workspace)
    c.idx[1, 2] = c.idx[1, 0]                 # twice: the weights are added
    c.idx[2, 1], c.idx[3, 0] = -5, 1 << 20
    c.idx[4] = torch.tensor([-1, 24, 1 << 30, -(1 << 31)])
    c.wt[0] = torch.tensor([0.0, -0.5, 2.0, 1e-30])
    y, y32 = c.given()
    c.check(y, y32, c.reference())
    st = c.layer.status()
    assert st["bad_expert_id"] == 6 and st["empty_rows"] == 1 and st["wait_timeout"] == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_nonfinite_values_stay_in_their_rows(kind):
    c = Case(kind, 5, E=24, k=4, seed=53)
    y, y32 = c.given()
    mb.moe_clear_device_status(c.layer.workspace)
    c.x[2, 7] = float("nan")
    z, z32 = c.given()
    rest = torch.tensor([0, 1, 3, 4], device="cuda")
    assert torch.equal(y32[rest], z32[rest]) and torch.isnan(z32[2]).all()
    assert c.layer.status()["nonfinite_output"] == c.H // 16
    # an expert with NaN weights poisons the rows that chose it alone
    c = Case(kind, 5, E=24, k=4, seed=53)
    e = int(c.idx[0, 1])
    for i, w in enumerate(c.raw[:3]):
        w[e].view(torch.uint8 if kind == "e4m3" else torch.int16).fill_(0x7F if kind == "e4m3" else 0x7FC0)
    z, z32 = c.given()
    hit = (c.idx == e).any(1)
    assert torch.isnan(z32[hit]).all() and torch.equal(z32[~hit], y32[~hit]) and bool((~hit).any())


@pytest.mark.parametrize("E,k", [(64, 5), (300, 8), (1000, 32), (40, 32)])
def test_equal_and_extreme_logits(E, k):
    """Rows of equal logits (the lowest ids), of a few values, and of infinities: the order and
    weights of moe_block_route."""
    c = Case("bf16", 4, E=E, k=k, I=64, Is=64, seed=70)
    c.router.zero_()
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    biases = [torch.zeros(E, device="cuda"), torch.arange(E, device="cuda").float() % 3,
              -torch.arange(E, device="cuda").float(), torch.full((E,), float("-inf"), device="cuda"),
              torch.full((E,), float("nan"), device="cuda"), torch.where(torch.arange(E, device="cuda") % 7 == 0, float("inf"), 0.0)]
    for bias in biases:
        y, y32, idx, wt = c.routed(bias)
        ri, rw = c.layer.route(c.x, off, bias[None])
        torch.cuda.synchronize()
        assert torch.equal(idx, ri) and torch.equal(wt.view(torch.int32), rw.view(torch.int32))


def test_nonfinite_logits_are_counted_once():
    c = Case("bf16", 3, E=16, k=4, seed=54)
    bias = torch.zeros(16, device="cuda")
    bias[3], bias[4] = float("-inf"), float("nan")
    mb.moe_clear_device_status(c.layer.workspace)
    y, y32, idx, wt = c.routed(bias)
    assert c.layer.status()["nonfinite_logits"] == 6
    assert not ((idx == 3) | (idx == 4)).any()
    c.check(y, y32, c.reference(idx, wt))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_repeat_same_bits_and_mixed_calls(kind):
    """Hundreds of calls in a row, both kinds, other sizes between: the barriers' flags are
    left ready for any next call."""
    c = Case(kind, 8, E=32, k=4, H=512, seed=55, max_rows=40)
    d = Case(kind, 2, E=16, k=2, H=256, seed=56, max_rows=8)
    d.layer.workspace = c.layer.workspace        # plans of other shapes may share a workspace
    y, y32, idx, wt = c.routed()
    g, g32 = c.given()
    f, f32 = d.given()
    p, p32, pi, pw = d.routed()
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    z = c.layer(c.x, off, 0.9).clone()
    for i in range(60):
        outs = [c.routed(), c.given(), d.given(), c.given(), d.routed()]
        zz = c.layer(c.x, off, 0.9).clone() if i % 7 == 0 else z
        outs.append(c.routed())
        torch.cuda.synchronize()
        assert torch.equal(outs[0][1], y32) and torch.equal(outs[0][2], idx) and torch.equal(outs[5][1], y32)
        assert torch.equal(outs[1][1], g32) and torch.equal(outs[3][1], g32)
        assert torch.equal(outs[2][1], f32) and torch.equal(outs[4][1], p32) and torch.equal(zz, z)
    c.status_clean()


def test_new_rows_every_call():
    """No result of an earlier call shows: other rows each time, back to back."""
    c = Case("bf16", 4, E=32, k=4, H=512, seed=57)
    xs = [randn(4, 512, seed=100 + i).to(BF) for i in range(20)]
    want = []
    for x in xs:
        c.x = x
        want.append(c.routed()[1].clone())
        torch.cuda.synchronize()
    ys = [torch.empty(4, 512, dtype=BF, device="cuda") for _ in xs]
    for x, y in zip(xs, ys):
        c.layer.token_pass(x, y=y)
    torch.cuda.synchronize()
    for y, w in zip(ys, want):
        assert torch.equal(y, w.to(BF))


def test_call_numbers_wrap():
    """The counter behind the logits' call numbers, set to shortly before their 32 bits wrap (a
    day's calls): rows that were never used before, and other rows each call."""
    c = Case("bf16", 8, E=32, k=4, H=512, seed=75)
    xs = [randn(8, 512, seed=300 + i).to(BF) for i in range(8)]
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    for start in ((1 << 32) - 4, (1 << 33) - 5, (1 << 53) - 4):
        c.layer.workspace.zero_()
        c.layer.workspace[1024:2048].view(torch.int64)[1] = start * 1024
        for i, x in enumerate(xs):
            R = 1 if i < 3 else 8
            c.x, c.R = x[:R].contiguous(), R
            y, y32, idx, wt = c.routed()
            ri, rw = c.layer.route(c.x, off if R == 8 else torch.tensor([0, 1], dtype=torch.int32, device="cuda"))
            torch.cuda.synchronize()
            assert torch.equal(idx, ri) and torch.equal(wt, rw)
            c.check(y, y32, c.reference(idx, wt))
        c.status_clean()


def test_in_place_and_rows_behind():
    c = Case("bf16", 3, seed=58)
    want = c.routed()[0]
    buf = torch.full((8, c.H), 2.0, dtype=BF, device="cuda")
    buf[:3] = c.x
    c.layer.token_pass(buf[:3], y=buf[:3])
    assert torch.equal(buf[:3], want) and torch.all(buf[3:] == 2)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_streams_and_graphs(kind):
    """On another stream, and two graphs over one workspace replayed in turn with eager calls."""
    c = Case(kind, 4, E=32, k=4, H=512, seed=59)
    base = [t.clone() for t in c.routed()]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    outs = c.routed(stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(base, outs))
    y1, y2 = torch.zeros_like(base[0]), torch.zeros_like(base[0])
    idx, wt = torch.zeros_like(base[2]), torch.zeros_like(base[3])
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1, stream=st):
        c.layer.token_pass(c.x, topk_idx=idx, topk_w=wt, y=y1)
    with torch.cuda.graph(g2, stream=st):
        c.layer.token_forward(c.x, idx, wt, y=y2)
    for i in range(10):
        c.x.copy_(randn(4, 512, seed=200 + i).to(BF))
        g1.replay()
        g2.replay()
        eager = c.routed()
        torch.cuda.synchronize()
        assert torch.equal(y1, eager[0]) and torch.equal(y2, eager[0]) and torch.equal(idx, eager[2])
    c.status_clean()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_wait_limit(kind):
    """With a limit of 1 ns the barriers' waits run out: the calls return, are counted, and the
    next ones are right again."""
    c = Case(kind, 4, E=32, k=4, H=512, seed=60)
    base, given = c.routed(), c.given()
    torch.cuda.synchronize()
    mb.moe_clear_device_status(c.layer.workspace)
    for _ in range(3):
        c.layer.plan.set_wait_limit(1)
        try:
            c.routed()
            c.given()
            torch.cuda.synchronize()
            st = c.layer.status()
        finally:
            c.layer.plan.set_wait_limit(0)
        assert st["wait_timeout"] > 0
        mb.moe_clear_device_status(c.layer.workspace)
        again, g2 = c.routed(), c.given()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(base, again))
        assert torch.equal(given[1], g2[1])
        c.status_clean()


def test_two_layers_on_two_streams():
    """Calls of two layers, each with its workspace, on two streams at once."""
    cs = [Case("bf16", 8, E=32, k=4, H=1024, I=512, Is=512, seed=71), Case("e4m3", 3, E=64, k=6, H=512, seed=72)]
    want = [c.routed() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [[], []]
    for _ in range(50):
        for c, st, o in zip(cs, streams, outs):
            with torch.cuda.stream(st):   # its outputs' memory is of the stream too
                o.append(c.routed())
    torch.cuda.synchronize()
    for c, w, o in zip(cs, want, outs):
        for got in o:
            assert all(torch.equal(a, b) for a, b in zip(w, got))
        c.status_clean()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_one_workspace_for_the_layer_and_the_products(kind):
    """The int8 and e4m3 products use the layer's workspace between its calls."""
    c = Case(kind, 4, E=32, k=4, H=512, seed=73, max_rows=2048)
    R, N, K = 520, 2048, 1024   # large enough for the tiles, whose x lies in the workspace
    need = mb.moe_i8_gemm_workspace_bytes(R, N, K)
    mem = c.layer.workspace
    assert 2 * R * K < need <= mem.numel()
    g = torch.Generator(device="cuda").manual_seed(1)
    xq = torch.randint(-127, 128, (R, K), generator=g, device="cuda").to(torch.int8)
    wq = torch.randint(-127, 128, (N, K), generator=g, device="cuda").to(torch.int8)
    xs, ws = torch.ones(R, device="cuda"), torch.ones(N, device="cuda")
    y = torch.empty(R, N, device="cuda")
    want = c.routed()
    for _ in range(5):
        mb.moe_i8_gemm(xq, xs, wq, ws, y, mem)
        got = c.routed()
        given = c.given(want[2], want[3])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)) and torch.equal(given[1], want[1])
        assert torch.equal(y.double(), xq.double() @ wq.double().t())
    c.status_clean()


def test_one_row_at_a_time_and_together():
    """Rows alone give what they give together, up to the order of fp32 sums; also a view of a
    larger batch, and R = 0."""
    c = Case("bf16", 8, E=48, k=6, H=768, seed=74)
    y, y32, idx, wt = c.routed()
    _, bound = c.reference(idx, wt)
    for r in range(8):
        a = torch.empty(1, c.H, dtype=BF, device="cuda")
        a32 = torch.empty(1, c.H, device="cuda")
        i1, w1 = torch.empty(1, 6, dtype=torch.int32, device="cuda"), torch.empty(1, 6, device="cuda")
        c.layer.token_pass(c.x[r:r + 1], topk_idx=i1, topk_w=w1, y=a, y_f32=a32)
        assert torch.equal(i1[0], idx[r]) and torch.equal(w1[0], wt[r])
        assert torch.all((a32[0] - y32[r]).abs() <= 2 * bound[r])
    none = c.layer.token_forward(c.x[:0], idx[:0], wt[:0])
    assert none.shape == (0, c.H)


FIRST = """
import torch
from sparse_moe_layer_row_gb300 import moe_block as mb
torch.manual_seed(0)
dev, BF = "cuda", torch.bfloat16
def w(*s): return (torch.randn(*s, device=dev) * 0.05).to(BF)
H, E, I, R, N = 256, 16, 128, 700, 2048
layer = mb.MoeBlockLayer(w(E, H), w(E, I, H), w(E, I, H), w(E, H, I), w(I, H), w(I, H), w(H, I), k=4, max_rows=8, max_blocks=1)
x, big, W = w(4, H), w(R, H), w(N, H)
n, y = torch.empty_like(x), torch.empty_like(x)
q, s = torch.empty(R, H, dtype=torch.int8, device=dev), torch.empty(R, device=dev)
wq, ws = torch.empty(N, H, dtype=torch.int8, device=dev), torch.empty(N, device=dev)
out = torch.empty(R, N, device=dev)
mem = torch.zeros(mb.moe_i8_gemm_workspace_bytes(R, N, H), dtype=torch.uint8, device=dev)
assert mem.numel() > 2 * R * H
def run():
    mb.moe_add_rmsnorm(x, None, 1e-6, residual=x, y=n)
    layer.token_pass(n, y=y)
    mb.moe_i8_quantize(big, q, s)
    mb.moe_i8_quantize(W, wq, ws)
    mb.moe_i8_gemm(q, s, wq, ws, out, mem)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    run()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (n, y, q, wq, out)]
for t in (n, y, q, wq, out): t.zero_()
run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (n, y, q, wq, out)))
assert out.abs().max() > 0 and not any(layer.status().values()) and not any(mb.moe_read_device_status(mem).values())
print("same")
"""


def test_first_calls_of_a_process_are_captured():
    """What a first call sets up (attributes, occupancy) is allowed inside a capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_scored_routing_into_the_layer():
    """Logits, routing by a rule, the experts in one kernel."""
    c = Case("e4m3", 5, E=32, k=4, H=512, seed=61)
    off = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    rule = mb.RouteRule(score="sigmoid", n_groups=4, top_groups=2, group_score="top2", scale=2.5)
    idx, w, _ = c.layer.route_scored(c.x, off, rule, select_bias=randn(32, seed=4, sigma=0.05))
    y, y32 = c.given(idx, w)
    c.check(y, y32, c.reference(idx, w))


def test_refusals():
    c = Case("bf16", 9, seed=62)
    L = c.layer
    with pytest.raises(mb.MoeError, match="at most 8"):
        c.given()
    with pytest.raises(mb.MoeError, match="at most 8"):
        c.routed()
    c = Case("bf16", 4, seed=62)
    L, y = c.layer, torch.empty(4, c.H, dtype=BF, device="cuda")
    for kw in (dict(idx=c.idx.long()), dict(idx=c.idx[:, :2].contiguous()), dict(wt=c.wt.double()), dict(x=c.x.float()),
               dict(x=c.x[:3])):
        with pytest.raises(ValueError):
            c.given(**kw)
    with pytest.raises(ValueError):
        L.token_pass(c.x, bias=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError):
        L.token_pass(c.x, y=y.float())
    with pytest.raises(mb.MoeError, match="workspace"):
        mb.moe_token_forward(L.plan, c.x, c.idx, c.wt, y, None, L.workspace[:1024])
    e = c.x[:0]
    assert L.token_pass(e).shape == (0, c.H)
    with pytest.raises(mb.MoeError, match="H="):
        Case("bf16", 1, H=8448, E=2, k=1, I=64, Is=64).given()
    w = W.TINY
    T = W.make_tensors(w, device="cuda")
    q = mb.MoeBlockLayer.quantized(T.w_router, W.quantize_experts(T, 8), k=w.k, max_rows=4, max_blocks=1)
    with pytest.raises(mb.MoeError, match="integer experts"):
        q.token_pass(T.x[:4].contiguous())


def test_a_decoding_step():
    """As a model runs them: norm with the residual, layer, norm with the residual and int8
    codes, projection, captured as one graph and replayed on new rows."""
    c = Case("e4m3", 3, E=32, k=4, H=512, seed=63)
    N = 256
    w1, w2 = (1 + 0.1 * randn(512, seed=1)).to(BF), (1 + 0.1 * randn(512, seed=2)).to(BF)
    wq, ws = torch.empty(N, 512, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    mb.moe_i8_quantize(randn(N, 512, seed=5, sigma=0.02), wq, ws)
    a, res = randn(3, 512, seed=6).to(BF), randn(3, 512, seed=7, sigma=3).to(BF)
    n1, y = torch.empty_like(a), torch.empty_like(a)
    q, s = torch.empty(3, 512, dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
    out = torch.empty(3, N, dtype=torch.float32, device="cuda")
    mem = torch.zeros(mb.moe_i8_gemm_workspace_bytes(3, N, 512), dtype=torch.uint8, device="cuda")
    stream = res.clone()

    def step():
        mb.moe_add_rmsnorm(a, w1, 1e-6, residual=stream, total=stream, y=n1)
        c.layer.token_pass(n1, y=y)
        mb.moe_add_rmsnorm(y, w2, 1e-6, residual=stream, total=stream, codes=q, scales=s)
        mb.moe_i8_gemm(q, s, wq, ws, out, mem)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    for i in range(4):
        a.copy_(randn(3, 512, seed=80 + i).to(BF))
        stream.copy_(res)
        step()
        torch.cuda.synchronize()
        eager = [t.clone() for t in (n1, y, q, s, out, stream)]
        stream.copy_(res)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, t) for p, t in zip(eager, (n1, y, q, s, out, stream)))
        # each step against 64 bits from the step before
        t1 = (a.float() + res.float()).to(BF).double()
        v = t1 * w1.double() * torch.rsqrt(t1.square().mean(1, keepdim=True) + 1e-6)
        assert torch.all((n1.double() - v).abs() <= 2.0 ** -7.9 * v.abs() + 1e-30)
        idx, wt = c.layer._topk_idx[:3], c.layer._topk_w[:3]
        want, bound = c.reference(idx, wt, n1)
        assert torch.all((y.double() - want).abs() <= bound + 2.0 ** -8 * (want.abs() + bound))
        acc = q.double() @ wq.double().t()
        ref = acc * s.double()[:, None] * ws.double()
        assert torch.all((out.double() - ref).abs() <= 2.0 ** -22 * ref.abs())
