"""Scored routing and e4m3 experts together, as one layer of a model runs them.

    python examples/scored_fp8_layer.py [--rows 32] [--passes 20]

The layer's router logits are routed by a rule (sigmoid scores, a selection bias,
the best groups of experts, renormalised weights with a scale), the experts are
e4m3 with one scale per 128 x 128 block, and a projection after the layer runs as
the dense product on quantised rows.  Prints the time of a pass and how far the
layer is from the same routing on its bf16 experts.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from sparse_moe_layer_row_gb300 import moe_block as mb, workloads as W


class ScoredFp8Layer:
    """Routing by a rule, e4m3 experts, and a projection [N, H] of the layer's output."""

    def __init__(self, T: W.Tensors, w_proj, k: int, rule: mb.RouteRule, select_bias,
                 max_rows: int, max_blocks: int):
        dev, (E, H) = T.w_router.device, T.w_router.shape
        self.moe = mb.MoeBlockLayer.fp8(T.w_router, W.fp8_experts(T), k, max_rows, max_blocks)
        self.rule, self.bias = rule, select_bias
        self.wq, self.ws = W.quantize_blocks_e4m3(w_proj)
        N = w_proj.shape[0]
        self.yq = torch.empty(max_rows, H, dtype=torch.float8_e4m3fn, device=dev)
        self.ys = torch.empty(H // 128 * max_rows, dtype=torch.float32, device=dev)
        self.out = torch.empty(max_rows, N, dtype=torch.bfloat16, device=dev)
        self.mem = torch.zeros(mb.moe_fp8_gemm_workspace_bytes(max_rows, N, H), dtype=torch.uint8,
                               device=dev)

    def __call__(self, x, block_offsets):
        R, H = x.shape
        idx, w, score = self.moe.route_scored(x, block_offsets, self.rule, select_bias=self.bias)
        # tau 1: every chosen expert is kept and the weights stay as they are; below 1 the
        # block's coreset by the experts' scores
        keep, _, wr, _ = self.moe.coreset(block_offsets, idx, w, 1.0, mass=score)
        y = self.moe.forward(x, block_offsets, idx, wr, keep)
        yq, ys, out = self.yq[:R], self.ys[:H // 128 * R].view(H // 128, R), self.out[:R]
        mb.moe_fp8_quantize(y, yq, ys)
        mb.moe_fp8_gemm(yq, ys, self.wq, self.ws, out, self.mem)
        return y, out


def main(argv=None) -> float:
    ap = argparse.ArgumentParser()
    ap.add_argument("--rows", type=int, default=32)
    ap.add_argument("--passes", type=int, default=20)
    ap.add_argument("--tiny", action="store_true", help="the tiny layer (256 wide, 16 experts)")
    args = ap.parse_args(argv)
    w = W.TINY if args.tiny else W.BLOCK32
    T = W.make_tensors(w, device="cuda")
    R = args.rows
    x = W.make_x(w, "cuda", rows=R, seed=5)
    nb = -(-R // 32)
    off = (torch.arange(nb + 1, device="cuda") * 32).clamp_max(R).to(torch.int32)
    rule = mb.RouteRule(score="sigmoid", n_groups=4, top_groups=2, group_score="top2", scale=2.5)
    bias = torch.linspace(-0.05, 0.05, w.E, device="cuda")
    proj = W.normal_bf16(7, 1, (w.H, w.H), 0.02, "cuda")
    layer = ScoredFp8Layer(T, proj, w.k, rule, bias, max_rows=R, max_blocks=nb)
    y, out = layer(x, off)
    # the same routing on the bf16 experts
    ref = mb.MoeBlockLayer(T.w_router, T.w_gate, T.w_up, T.w_down, T.ws_gate, T.ws_up, T.ws_down,
                           k=w.k, max_rows=R, max_blocks=nb)
    idx, wt, score = ref.route_scored(x, off, rule, select_bias=bias)
    keep, _, wr, _ = ref.coreset(off, idx, wt, 1.0, mass=score)
    yr = ref.forward(x, off, idx, wr, keep)
    rel = float((y.float() - yr.float()).norm() / yr.float().norm())
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    for _ in range(args.passes):
        layer(x, off)
    b.record()
    torch.cuda.synchronize()
    print(f"{R} rows, {w.E} experts: {a.elapsed_time(b) * 1e3 / args.passes:.1f} us a pass; "
          f"e4m3 against bf16 experts: {rel:.4f} of the output's norm; "
          f"projection {tuple(out.shape)} finite: {bool(torch.isfinite(out).all())}")
    return rel


if __name__ == "__main__":
    main()
