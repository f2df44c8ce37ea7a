"""The router, the products, the 8-bit checkpoint and the int8 products together, as a layer uses them: every step
against its formula on the inputs that it had, the layer's gradients against 64-bit ones, and the example.

A gradient of the layer goes through at most ten roundings to bf16 (rows, h, y, out rows, d_rows, dy, dh and the
recomputed y among them), each of at most 2^-8 of a value, so of a tensor's norm; products of random matrices pass
a relative error on as it is: 10 * 2^-8 = 0.04 of the norm."""

import os
import sys

import pytest
import torch

import block_scaled_grouped_amd as bsg
from gpu_util import device

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import routed_experts  # noqa: E402

pytestmark = pytest.mark.gpu

F64 = torch.float64
BOUND = 10 * 2.0 ** -8


def _decoded(data, scales):
    d = data.cpu().view(torch.float8_e4m3fn).to(torch.float32).to(F64)
    s = torch.exp2(scales.cpu().to(F64) - 127)
    return (d.view(d.shape[0], -1, 32) * s[:, :, None]).view(d.shape)


class _Gate(torch.autograd.Function):
    """weight silu(g) u, with the derivatives at the kept values of [g | u]."""

    @staticmethod
    def forward(ctx, h, w, kept):
        ctx.save_for_backward(w, kept)
        f = h.shape[1] // 2
        return w[:, None] * torch.nn.functional.silu(h[:, :f]) * h[:, f:]

    @staticmethod
    def backward(ctx, dy):
        w, kept = ctx.saved_tensors
        f = kept.shape[1] // 2
        g, u, s = kept[:, :f], kept[:, f:], torch.sigmoid(kept[:, :f])
        dh = torch.cat([dy * w[:, None] * u * s * (1 + g * (1 - s)), dy * w[:, None] * g * s], 1)
        return dh, (dy * g * s * u).sum(1), None


def _reference(layer, x, saved, d_out, mask):
    """Gradients of router, w1 and w2 in 64 bits on the host, for the experts that were chosen; the second product's
    weight gradient takes the activation at the kept values."""
    _, _, _, r, held, token, _, offsets, _, data, scales = saved
    experts, held, token, off = (t.cpu() for t in (r["experts"], held, token, offsets))
    kept = _decoded(data, scales)
    x, d_out = x.cpu().to(F64), d_out.cpu().to(F64)
    router, w1, w2 = (t.detach().cpu().to(F64).requires_grad_() for t in (layer.router, layer.w1, layer.w2))
    p = torch.softmax(x @ router, 1)
    live = torch.ones(x.shape[0], dtype=torch.bool) if mask is None else mask.cpu()
    w = p.gather(1, experts.long().clamp(min=0))
    w = (w / w.sum(1, keepdim=True)).flatten()[held]
    counts, n = r["counts"].cpu().to(F64), int(live.sum())
    balance = layer.experts / (layer.k * n * n) * (counts * p[live].sum(0)).sum()
    out = torch.zeros_like(x)
    f = layer.w2.shape[2]
    d_w2 = torch.zeros_like(w2)
    for e in range(layer.experts):
        rows = slice(int(off[e]), int(off[e + 1]))
        h = x[token[rows]] @ w1[e].t()
        y = _Gate.apply(h, w[rows], kept[rows])
        out = out.index_add(0, token[rows], y @ w2[e].t())
        k = kept[rows]
        again = w[rows].detach()[:, None] * torch.nn.functional.silu(k[:, :f]) * k[:, f:]
        d_w2[e] = d_out[token[rows]].t() @ again
    (out * d_out).sum().add(float(layer.balance) * balance).backward()
    return out.detach(), float(balance.detach()), (router.grad, w1.grad, d_w2)


def _near(got, want, what):
    got = got.detach().cpu().to(F64)
    off = float((got - want).norm() / want.norm())
    assert off <= BOUND, (what, off)


@pytest.mark.parametrize("tokens,experts,k,width,hidden,masked", [(300, 8, 2, 128, 160, 0), (1000, 5, 3, 64, 512, 100),
                                                                  (7, 16, 4, 256, 32, 1), (1, 4, 1, 64, 96, 0)])
def test_layer_gradients(tokens, experts, k, width, hidden, masked):
    layer = routed_experts.RoutedExperts(experts, k, width, hidden, device(), balance=0.5)
    gen = torch.Generator().manual_seed(tokens)
    x = torch.randn((tokens, width), generator=gen).to(torch.bfloat16).to(device())
    mask = None
    if masked:
        mask = torch.ones(tokens, dtype=torch.bool)
        mask[torch.randperm(tokens, generator=gen)[:masked]] = False
        mask = mask.to(device())
    d_out = torch.randn((tokens, width), generator=gen).to(device()) / tokens
    out, balance, saved = layer.forward(x, mask)
    grads = layer.backward(d_out, saved)
    assert int(layer.status) == 0
    want_out, want_balance, want = _reference(layer, x, saved, d_out, mask)
    _near(out, want_out, "out")
    assert abs(float(balance) - want_balance) <= 1e-4 * want_balance
    for got, ref, name in zip(grads, want, ("router", "w1", "w2")):
        _near(got, ref, name)
    if mask is not None:
        assert bool((out[~mask] == 0).all())


@pytest.mark.parametrize("tokens,experts,k,width,hidden", [(1, 8, 2, 256, 512), (40, 8, 2, 256, 512), (900, 4, 2, 128, 96)])
def test_serving(tokens, experts, k, width, hidden):
    """Against the same layer in 64 bits on the dequantized weights: a token's integer is off by half a step of its
    row's largest / 127, some 2^-9 of the row's norm in the mean and 2^-6 at most for normal rows, twice."""
    layer = routed_experts.RoutedExperts(experts, k, width, hidden, device())
    x = torch.randn((tokens, width), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(device())
    weights = layer.quantized()
    out = layer.serve(x, weights).cpu().to(F64)
    w1, w2 = ((q.cpu().to(F64) * s.cpu().to(F64)[:, :, None]) for q, s in weights)
    r = bsg.moe_router_topk(x.float() @ layer.router, k)
    xs, want = x.cpu().to(F64), torch.zeros((tokens, width), dtype=F64)
    for j in range(k):
        for t in range(tokens):
            e, w = int(r["experts"][t, j]), float(r["weights"][t, j])
            h = w1[e] @ xs[t]
            want[t] += w2[e] @ (w * torch.nn.functional.silu(h[:hidden]) * h[hidden:])
    assert float((out - want).norm() / want.norm()) <= 2 * 2.0 ** -6 + 4 * 2.0 ** -8


def test_serving_step_in_a_graph():
    """Router, activation and int8 products captured together and replayed on new tokens (the rows' order is
    fixed: every token goes to all experts)."""
    experts, tokens, width, hidden = 4, 6, 128, 64
    layer = routed_experts.RoutedExperts(experts, experts, width, hidden, device())
    (q1, s1), (q2, s2) = layer.quantized()
    xs = [torch.randn((tokens, width), device=device()).to(torch.bfloat16) for _ in range(2)]
    rows = tokens * experts
    offsets = torch.arange(experts + 1, device=device()) * tokens
    spaces = [bsg.grouped_gemm_int8_dynamic_workspace(rows, max(width, hidden)) for _ in range(2)]
    router_space = bsg.moe_router_topk_workspace(tokens, experts)

    def step(x, ws):
        r = bsg.moe_router_topk(x.float() @ layer.router, experts, workspace=router_space)
        # weight of token t and expert e, expert by expert
        w = torch.zeros((tokens, experts), device=device()).scatter(1, r["experts"].long(), r["weights"])
        h = bsg.grouped_gemm_int8_dynamic(x.repeat(experts, 1), q1, s1, offsets, workspace=ws[0])
        y, _, _ = bsg.grouped_swiglu_checkpoint_mxfp8(h, offsets, row_weights=w.t().contiguous().flatten(), keep=False)
        return bsg.grouped_gemm_int8_dynamic(y, q2, s2, offsets, workspace=ws[1])

    want = [step(x, spaces).clone() for x in xs]
    x = xs[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x, spaces)
    for i in (1, 0, 1):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want[i])


def test_example_runs():
    layer, losses, balances = routed_experts.train(steps=2, experts=4, width=64, hidden=64, tokens=128)
    assert all(v == v and v < float("inf") for v in losses + balances)
    out = layer.serve(torch.randn((3, 64), device=device()).to(torch.bfloat16), layer.quantized())
    assert out.shape == (3, 64) and bool(out.isfinite().all())
