"""The 16-bit operators together, as a training step and a serving step use them.

Training: a two-layer mixture of experts whose weights a low-precision recipe leaves in bf16.  Rows are sorted
by expert; forward, data gradients and weight gradients (added into float32 main gradients over two
micro-batches) are grouped products; the main gradients are clipped by their global norm; SGD on float32
master weights.

Serving: requests of different lengths, prompts and single tokens, go through one projection beside the
adapters that they ask for.

    python examples/adapted_experts.py [--steps 20]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_grouped_amd as bsg  # noqa: E402


def route(x, router, experts):
    """Rows sorted by expert (one expert a row) and the groups' offsets."""
    choice = (x.float() @ router).argmax(1)
    order = torch.argsort(choice, stable=True)
    sizes = torch.bincount(choice, minlength=experts).to(torch.int32)
    return x[order].contiguous(), bsg.group_offsets_i32_to_i64(sizes)[1]


class Experts:
    """y = relu(x W1_e^T) W2_e^T with float32 master weights and main gradients."""

    def __init__(self, experts, width, hidden, device, seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.master = [torch.randn((experts, hidden, width), generator=gen, device=device) * width ** -0.5,
                       torch.randn((experts, width, hidden), generator=gen, device=device) * hidden ** -0.5]
        self.main_grads = [torch.zeros_like(m) for m in self.master]
        self.plan = bsg.grad_clip_plan(self.main_grads)       # clips in place
        self.workspace = bsg.gemm_workspace(device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def micro_batch(self, x, target, offsets, rows):
        """Adds the micro-batch's gradients of sum((y - target)^2) / rows; returns the loss."""
        mm = lambda *a, **k: bsg.grouped_gemm_16bit(*a, offsets, workspace=self.workspace,  # noqa: E731
                                                    status=self.status, **k)
        w1, w2 = (m.to(torch.bfloat16) for m in self.master)
        h = mm(bsg.BSG_FPROP_TN, x, w1).relu_()
        diff = mm(bsg.BSG_FPROP_TN, h, w2, out_dtype=bsg.BSG_OUT_F32) - target
        dy = (diff * (2.0 / rows)).to(torch.bfloat16)
        dh = mm(bsg.BSG_DGRAD_NN, dy, w2).mul_(h > 0)
        mm(bsg.BSG_WGRAD_NT, dy, h, c=self.main_grads[1], out=self.main_grads[1])
        mm(bsg.BSG_WGRAD_NT, dh, x, c=self.main_grads[0], out=self.main_grads[0])
        return diff.square().sum() / rows

    def update(self, lr, max_norm):
        norm = bsg.clip_grad_norm(self.plan, max_norm, status=self.status)
        for m, g in zip(self.master, self.main_grads):
            m.add_(g, alpha=-lr)
            g.zero_()
        return norm


def train(steps=20, experts=8, width=256, hidden=512, rows=1024, lr=0.5, max_norm=1.0, device="cuda"):
    """Losses and gradient norms of `steps` steps of two micro-batches each."""
    gen = torch.Generator(device=device).manual_seed(1)
    model = Experts(experts, width, hidden, device)
    router = torch.randn((width, experts), generator=gen, device=device)
    teacher = torch.randn((width, width), generator=gen, device=device) * width ** -0.5
    batches = []
    for _ in range(2):
        x, offsets = route(torch.randn((rows, width), generator=gen, device=device).to(torch.bfloat16), router,
                           experts)
        batches.append((x, x.float() @ teacher, offsets))
    losses, norms = [], []
    for _ in range(steps):
        loss = sum(model.micro_batch(x, t, o, 2 * rows) for x, t, o in batches)
        norms.append(model.update(lr, max_norm))
        losses.append(loss)
    if int(model.status):
        raise RuntimeError("device status %d" % int(model.status))
    return [float(v) for v in losses], [float(v) for v in norms]


def serve(lengths=(37, 1, 1, 120, 1), adapters=(0, 2, -1, 1, 2), width=512, out=1024, rank=16, device="cuda"):
    """The projection of a batch of requests, each with its adapter (-1: none)."""
    gen = torch.Generator(device=device).manual_seed(2)
    bf16 = dict(generator=gen, device=device)
    count = max(adapters) + 1
    sizes = torch.tensor(lengths, dtype=torch.int32, device=device)
    offsets = bsg.group_offsets_i32_to_i64(sizes)[1]
    x = torch.randn((sum(lengths), width), **bf16).to(torch.bfloat16)
    w = (torch.randn((out, width), **bf16) * width ** -0.5).to(torch.bfloat16)
    lora_a = (torch.randn((count, rank, width), **bf16) * width ** -0.5).to(torch.bfloat16)
    lora_b = (torch.randn((count, out, rank), **bf16) * 0.1).to(torch.bfloat16)
    scale = torch.full((count,), 2.0, device=device)
    ids = torch.tensor(adapters, dtype=torch.int32, device=device)
    workspace = bsg.grouped_lora_gemm_16bit_workspace(x.shape[0], out, width, rank, device)
    y = bsg.grouped_lora_gemm_16bit(x, w, lora_a, lora_b, offsets, ids, scale, workspace=workspace)
    return y, (x, w, lora_a, lora_b, scale)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    args = ap.parse_args()
    losses, norms = train(args.steps)
    for i, (l, n) in enumerate(zip(losses, norms)):
        print("step %2d  loss %8.4f  gradient norm %8.4f" % (i, l, n))
    y, _ = serve()
    print("served %d rows of %d columns" % y.shape)


if __name__ == "__main__":
    main()
