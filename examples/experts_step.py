"""One training step of a layer of experts in 8 bits, on the package's operators.

Tokens choose experts, an expert's rows go through its matrix, and each token gets the
weighted sum of its rows back; then every gradient. Activations and weights are e4m3,
gradients e5m2, with block scales; the weights' codes in 128 x 128 blocks serve the forward
product and, transposed in place, the gradient of the activations.

    python examples/experts_step.py [--tokens 4096 --experts 64 --top-k 8 --inputs 2048 --outputs 1024]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_06_amd as dg  # noqa: E402

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


def quantize_experts(weights):
    """The experts' matrices (E, N, K) as a BlockTensor in 128 x 128 blocks."""
    parts = [dg.gemm_block_quantize_tensors(w, E4, dg.BLOCK)[0] for w in weights]
    return dg.BlockTensor(torch.stack([p.data for p in parts]), torch.stack([p.scale for p in parts]), dg.BLOCK)


def forward(x, logits, router, bias, W):
    """(out, saved): out (T, N) from tokens x (T, K), their logits (T, E) and the experts' W (E, N, K)."""
    index, weight = dg.gemm_experts_route_tensors(logits, router, bias)
    plan = dg.gemm_experts_dispatch_tensors(index, W.data.shape[0], dg.BLOCK)
    codes, _ = dg.gemm_block_quantize_tensors(x, E4)
    y = dg.gemm_experts_product_tensors(codes, W, plan, x.dtype)
    return dg.gemm_experts_combine_tensors(y, plan, weight), (x, logits, router, W, index, weight, plan, y)


def backward(saved, grad):
    """Gradients of x, of the logits and of the experts' matrices (float32) from that of out."""
    x, logits, router, W, index, weight, plan, y = saved
    y_grad, weight_grad = dg.gemm_experts_combine_backward_tensors(y, plan, weight, grad)
    rows, columns = dg.gemm_block_quantize_tensors(y_grad, E5, transposed=True)
    x_rows = dg.gemm_experts_product_tensors(rows, W.t(), plan, x.dtype, gather=False)
    x_grad = dg.gemm_experts_combine_tensors(x_rows, plan, torch.ones_like(weight))
    _, inputs = dg.gemm_block_quantize_tensors(x, E4, natural=False, transposed=True, rows=plan.rows)
    W_grad = dg.gemm_experts_gradient_tensors(columns, inputs, plan)
    return x_grad, dg.gemm_experts_route_backward_tensors(logits, router, index, weight_grad), W_grad


def plain(x, logits, index, W, grad):
    """out and the same gradients from full-precision numbers, float32, for the given choice."""
    x, logits, W = (t.float().requires_grad_(True) for t in (x, logits, W))
    p = torch.sigmoid(logits).gather(1, index.long())
    w = p / p.sum(1, keepdim=True)
    out = torch.zeros(x.shape[0], W.shape[1], device=x.device)
    for e in range(W.shape[0]):
        t, slot = (index == e).nonzero(as_tuple=True)
        out = out.index_add(0, t, (x[t] @ W[e].t()) * w[t, slot][:, None])
    out.backward(grad.float())
    return out.detach(), x.grad, logits.grad, W.grad


def main(tokens=4096, experts=64, top_k=8, inputs=2048, outputs=1024, seed=0, repeat=10):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, logits = normal(tokens, inputs).bfloat16(), normal(tokens, experts)
    full = normal(experts, outputs, inputs) * inputs ** -0.5
    W, grad = quantize_experts(full), normal(tokens, outputs).bfloat16()
    router = dg.router(top_k, "sigmoid", renorm=True)
    bias = 0.1 * normal(experts)

    def step():
        out, saved = forward(x, logits, router, bias, W)
        return out, saved, backward(saved, grad)

    out, saved, grads = step()
    want = plain(x, logits, saved[4], full, grad)
    off = {n: float((a.float() - b).norm() / b.norm())
           for n, a, b in zip(("out", "x_grad", "logits_grad", "W_grad"), (out, *grads), want)}
    torch.cuda.synchronize()
    start, end = torch.cuda.Event(True), torch.cuda.Event(True)
    start.record()
    for _ in range(repeat):
        step()
    end.record()
    torch.cuda.synchronize()
    ms = start.elapsed_time(end) / max(repeat, 1)
    rate = 6 * tokens * top_k * inputs * outputs / ms / 1e9
    print(f"{tokens} tokens x {top_k} of {experts} experts, {inputs} -> {outputs}: {ms:.3f} ms a step, "
          f"{rate:.0f} TFLOP/s in the products; off full precision by "
          + ", ".join(f"{n} {v:.3f}" for n, v in off.items()))
    return off


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("experts", 64), ("top-k", 8), ("inputs", 2048), ("outputs", 1024)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    main(a.tokens, a.experts, a.top_k, a.inputs, a.outputs)
