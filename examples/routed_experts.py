"""A routed layer of gated experts, as a training step and a serving step use it.

Training: a router picks the experts of every token and balances them; the experts' rows go through two grouped
products with a gated activation between them, whose input is kept in 8 bits for the backward pass; the gradients
go back through the products, the activation and the router.

Serving: the same layer with the experts' weights in 8-bit integers, a scale for each channel, and the tokens
quantized on the way.

    python examples/routed_experts.py [--steps 20]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_grouped_amd as bsg  # noqa: E402


def by_expert(experts, counts):
    """Slots of `experts` [tokens, k] in the experts' order, and the offsets of their groups.  Slots without an
    expert (-1) come first and are left out."""
    order = torch.argsort(experts.flatten(), stable=True)
    held = order[experts.numel() - int(counts.sum()):]
    return held, bsg.group_offsets_i32_to_i64(counts)[1]


class RoutedExperts:
    """out[t] = sum over t's experts e of  w2_e (weight silu(g) u),  [g | u] = w1_e x_t."""

    def __init__(self, experts, k, width, hidden, device, balance=0.01, seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        normal = lambda *shape: torch.randn(shape, generator=gen, device=device)  # noqa: E731
        self.k, self.experts = k, experts
        self.router = normal(width, experts) * width ** -0.5
        self.w1 = (normal(experts, 2 * hidden, width) * width ** -0.5).to(torch.bfloat16)
        self.w2 = (normal(experts, width, hidden) * hidden ** -0.5).to(torch.bfloat16)
        self.workspace = bsg.gemm_workspace(device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.balance = torch.full((1,), balance, device=device)

    def _mm(self, mode, a, b, offsets, **kw):
        return bsg.grouped_gemm_16bit(mode, a, b, offsets, workspace=self.workspace, status=self.status, **kw)

    def forward(self, x, mask=None):
        """(out [tokens, width] float32, the balance loss, what the backward pass needs)"""
        logits = x.float() @ self.router
        r = bsg.moe_router_topk(logits, self.k, mask=mask, status=self.status)
        held, offsets = by_expert(r["experts"], r["counts"])
        token = held // self.k
        rows = x[token]
        h = self._mm(bsg.BSG_FPROP_TN, rows, self.w1, offsets)
        weights = r["weights"].flatten()[held]
        y, data, scales = bsg.grouped_swiglu_checkpoint_mxfp8(h, offsets, row_weights=weights, status=self.status)
        out_rows = self._mm(bsg.BSG_FPROP_TN, y, self.w2, offsets)
        out = torch.zeros_like(x, dtype=torch.float32).index_add_(0, token, out_rows.float())
        return out, r["loss"], (x, mask, logits, r, held, token, rows, offsets, weights, data, scales)

    def backward(self, d_out, saved):
        """Gradients of router, w1 and w2 for d_out [tokens, width] and the balance loss."""
        x, mask, logits, r, held, token, rows, offsets, weights, data, scales = saved
        d_rows = d_out[token].to(torch.bfloat16)
        dy = self._mm(bsg.BSG_DGRAD_NN, d_rows, self.w2, offsets)
        dh, d_weight, y = bsg.grouped_swiglu_checkpoint_mxfp8_backward(
            data, scales, dy, offsets, row_weights=weights, recompute=True, status=self.status)
        d_w2 = self._mm(bsg.BSG_WGRAD_NT, d_rows, y, offsets, out_dtype=bsg.BSG_OUT_F32)
        d_w1 = self._mm(bsg.BSG_WGRAD_NT, dh, rows, offsets, out_dtype=bsg.BSG_OUT_F32)
        d_weights = torch.zeros_like(r["weights"])
        d_weights.view(-1)[held] = d_weight
        d_logits = bsg.moe_router_topk_backward(logits, r["experts"], r["counts"], r["live"], d_weights=d_weights,
                                                d_loss=self.balance, mask=mask)
        return x.float().t() @ d_logits, d_w1, d_w2

    def quantized(self):
        """The experts' weights in 8-bit integers: ((w1, scales), (w2, scales))."""
        out = []
        for w in (self.w1, self.w2):
            q, s = bsg.grouped_quantize_int8(w.view(-1, w.shape[2]))
            out.append((q.view(w.shape), s.view(w.shape[:2])))
        return out

    def serve(self, x, weights):
        """out [tokens, width] from the quantized weights."""
        r = bsg.moe_router_topk(x.float() @ self.router, self.k)
        held, offsets = by_expert(r["experts"], r["counts"])
        token = held // self.k
        h = bsg.grouped_gemm_int8_dynamic(x[token], *weights[0], offsets, status=self.status)
        y, _, _ = bsg.grouped_swiglu_checkpoint_mxfp8(h, offsets, row_weights=r["weights"].flatten()[held], keep=False)
        out_rows = bsg.grouped_gemm_int8_dynamic(y, *weights[1], offsets, status=self.status)
        return torch.zeros_like(x, dtype=torch.float32).index_add_(0, token, out_rows.float())


def train(steps=20, experts=8, k=2, width=256, hidden=512, tokens=1024, lr=0.3, device="cuda"):
    """Losses of `steps` steps towards a linear teacher, and the balance losses."""
    gen = torch.Generator(device=device).manual_seed(1)
    layer = RoutedExperts(experts, k, width, hidden, device)
    master = [layer.w1.float(), layer.w2.float()]
    x = torch.randn((tokens, width), generator=gen, device=device).to(torch.bfloat16)
    target = x.float() @ (torch.randn((width, width), generator=gen, device=device) * width ** -0.5)
    losses, balances = [], []
    for _ in range(steps):
        out, balance, saved = layer.forward(x)
        diff = out - target
        d_router, d_w1, d_w2 = layer.backward(diff * (2.0 / tokens), saved)
        layer.router -= lr * d_router
        for m, d in zip(master, (d_w1, d_w2)):
            m -= lr * d
        layer.w1, layer.w2 = (m.to(torch.bfloat16) for m in master)
        losses.append(diff.square().sum() / tokens)
        balances.append(balance)
    if int(layer.status):
        raise RuntimeError("device status %d" % int(layer.status))
    return layer, [float(v) for v in losses], [float(v) for v in balances]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    args = ap.parse_args()
    layer, losses, balances = train(args.steps)
    for i, (loss, balance) in enumerate(zip(losses, balances)):
        print("step %2d  loss %8.4f  balance %7.4f" % (i, loss, balance))
    x = torch.randn((5, layer.w2.shape[1]), device="cuda").to(torch.bfloat16)
    print("served %d tokens of %d columns" % layer.serve(x, layer.quantized()).shape)


if __name__ == "__main__":
    main()
