"""A mixture-of-experts feed-forward layer in FP8: training steps and a decode step.

    python examples/moe_layer.py [--tokens 2048] [--steps 20]

Every expert computes y = (u g / (1 + exp(-g))) W2^T with [g | u] = x W13^T.  The
layer keeps nothing between its passes but 8-bit operands: the quantised tokens,
the gated activation's checkpoint and its result.

  forward   sort -> permute + quantise -> product -> gated activation -> product -> combine
  backward  combine's gradient -> product -> gated activation's gradient -> product -> combine,
            and a weight gradient for each product
"""
import argparse
import os
import sys
from typing import NamedTuple

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from moe_grouped_gemm_block_amd import dg


class Weights(NamedTuple):
    """[E][N][K] weights in 8 bits with 128 x 128 scales, and the same transposed
    for the gradient with respect to the input (a block's transpose has its scale)."""
    q: torch.Tensor
    s: torch.Tensor
    qt: torch.Tensor
    st: torch.Tensor


def quantise_weights(w):
    E, N, K = w.shape
    q, s = dg.quantize_fp8_blockscaled(w.reshape(E * N, K), 128)
    q, s = q.view(E, N, K), s.view(E, N // 128, K // 128)
    return Weights(q, s, q.transpose(1, 2).contiguous(), s.transpose(1, 2).contiguous())


class MoELayer:
    """hidden and inner are multiples of 128.  The master weights w13
    [E][2 inner][hidden] and w2 [E][hidden][inner] are float32."""

    def __init__(self, experts, hidden, inner, device="cuda", generator=None):
        self.experts, self.hidden, self.inner = experts, hidden, inner
        self.w13 = torch.randn(experts, 2 * inner, hidden, device=device, generator=generator) * hidden ** -0.5
        self.w2 = torch.randn(experts, hidden, inner, device=device, generator=generator) * inner ** -0.5
        self.refresh()

    def refresh(self):
        """The 8-bit weights from the master weights."""
        self.q13, self.q2 = quantise_weights(self.w13), quantise_weights(self.w2)

    def forward(self, x, ids, weights):
        """out [T][hidden] and what backward needs, for tokens x (bfloat16), expert
        ids [T][k] and router weights [T][k] (float32)."""
        plan = dg.moe_sort(ids, self.experts)
        xq, sx = dg.moe_permute_fp8(x, plan.slot_row, plan.row_slot)
        h = dg.grouped_gemm_fp8(xq, sx, self.q13.q, self.q13.s, plan.group_offsets, group_counts=plan.group_counts)
        a, sa, hq, sh = dg.swiglu_fp8(h)
        y = dg.grouped_gemm_fp8(a, sa, self.q2.q, self.q2.s, plan.group_offsets, group_counts=plan.group_counts)
        out = dg.moe_combine(y, plan.slot_row, weights)
        return out, (plan, weights, xq, sx, a, sa, hq, sh, y)

    def backward(self, dout, saved):
        """Gradients (dx, dweights, dw13, dw2) of dout (bfloat16)."""
        plan, weights, xq, sx, a, sa, hq, sh, y = saved
        offs, counts = plan.group_offsets, plan.group_counts
        dy, dweights = dg.moe_combine_bwd(dout, y, plan.slot_row, plan.row_slot, weights)
        dw2 = dg.grouped_wgrad_fp8(dy, a, sa, offs, counts)
        da = dg.grouped_gemm_fp8(*dg.quantize_fp8_blockscaled(dy, 1), self.q2.qt, self.q2.st, offs, group_counts=counts)
        dh = dg.swiglu_fp8_bwd(da, hq, sh)
        dw13 = dg.grouped_wgrad_fp8(dh, xq, sx, offs, counts)
        drows = dg.grouped_gemm_fp8(*dg.quantize_fp8_blockscaled(dh, 1), self.q13.qt, self.q13.st, offs,
                                    group_counts=counts)
        return dg.moe_combine(drows, plan.slot_row), dweights, dw13, dw2

    def decode(self, x, ids, weights):
        """The forward pass for a few tokens: packed segments, no checkpoint."""
        plan = dg.moe_sort(ids, self.experts, align=1)
        xq, sx = dg.moe_permute_fp8(x, plan.slot_row, plan.row_slot)
        h = dg.grouped_gemm_fp8_segments(xq, sx, self.q13.q, self.q13.s, plan.group_offsets)
        a, sa, _, _ = dg.swiglu_fp8(h, checkpoint=False)
        y = dg.grouped_gemm_fp8_segments(a, sa, self.q2.q, self.q2.s, plan.group_offsets)
        return dg.moe_combine(y, plan.slot_row, weights)


def route(x, router, k):
    """Expert ids and router weights: the k largest logits, softmax over them."""
    top = torch.topk(x.float() @ router, k, dim=1)
    return top.indices, torch.softmax(top.values, dim=1)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--top-k", type=int, default=2)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=1024)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=0.05)
    args = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)
    layer = MoELayer(args.experts, args.hidden, args.inner, generator=g)
    teacher = MoELayer(args.experts, args.hidden, args.inner, generator=g)
    router = torch.randn(args.hidden, args.experts, device="cuda", generator=g) * args.hidden ** -0.5
    x = torch.randn(args.tokens, args.hidden, device="cuda", generator=g).bfloat16()
    ids, weights = route(x, router, args.top_k)
    target = teacher.forward(x, ids, weights)[0].float()
    for step in range(args.steps):
        out, saved = layer.forward(x, ids, weights)
        diff = out.float() - target
        _, _, dw13, dw2 = layer.backward((diff / args.tokens).bfloat16(), saved)
        layer.w13 -= args.lr * args.experts * dw13
        layer.w2 -= args.lr * args.experts * dw2
        layer.refresh()
        print(f"step {step}: loss {0.5 * float(diff.square().sum()) / args.tokens:.4f}", flush=True)
    few = min(4, args.tokens)
    one = layer.decode(x[:few].contiguous(), ids[:few].contiguous(), weights[:few].contiguous())
    whole = layer.forward(x, ids, weights)[0][:few]
    err = float((one.float() - whole.float()).norm() / whole.float().norm())
    print(f"decode of {few} tokens: relative difference from the whole batch {err:.2e}")


if __name__ == "__main__":
    main()
