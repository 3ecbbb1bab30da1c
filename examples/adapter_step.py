"""One fine-tuning step of adapters around a gated layer, on the package's operators.

Requests with adapters of their own go through one shared layer: a projection to a gate and
its values, the gated activation, a projection back, and the loss over the vocabulary. The
shared weights are frozen; the adapters' gradients and the gradient of the input come back.
Neither the logits nor the activations are kept whole: the loss takes the vocabulary in
pieces, and what the backward pass needs of the activation's input is held in 8 bits.

    python examples/adapter_step.py [--tokens 4096 --adapters 4 --rank 16 --width 2048 --inner 4096 --words 32768]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_06_amd as dg  # noqa: E402

E4 = torch.float8_e4m3fn


def forward(x, p, index, target):
    """(loss, saved) of x (T, K), parameters p and each row's adapter and next word."""
    z, u_in = dg.gemm_adapters_tensors(x, p["w_in"], p["a_in"], p["b_in"], index, p["scale"], keep=True)
    y, codes = dg.gemm_activation_tensors(z, "silu", True, E4)
    h, u_out = dg.gemm_adapters_tensors(y, p["w_out"], p["a_out"], p["b_out"], index, p["scale"], keep=True)
    loss, lse = dg.gemm_loss_tensors(h, p["head"], target)
    return loss, (x, p, index, target, u_in, codes, u_out, h, lse)


def backward(saved, grad):
    """Gradients of x and of the adapters from grad (T), that of the loss."""
    x, p, index, target, u_in, codes, u_out, h, lse = saved
    plan = dg.gemm_experts_dispatch_tensors(index[:, None].contiguous(), p["a_in"].shape[0])
    h_grad, _ = dg.gemm_loss_backward_tensors(grad, h, p["head"], target, lse, w_grad=False)
    y = dg.gemm_activation_value_tensors(codes, "silu", True, h.dtype)
    y_grad, a_out, b_out = dg.gemm_adapters_backward_tensors(h_grad, y, u_out, p["w_out"], p["a_out"], p["b_out"],
                                                             index, plan, p["scale"])
    z_grad, _ = dg.gemm_activation_backward_tensors(y_grad, codes, "silu", True, value=False)
    x_grad, a_in, b_in = dg.gemm_adapters_backward_tensors(z_grad, x, u_in, p["w_in"], p["a_in"], p["b_in"], index,
                                                           plan, p["scale"])
    return {"x": x_grad, "a_in": a_in, "b_in": b_in, "a_out": a_out, "b_out": b_out}


def plain(x, p, index, target, grad):
    """loss and the same gradients from full-precision numbers, float32."""
    p = {n: t.float() for n, t in p.items()}
    x = x.float().requires_grad_(True)
    leaves = {n: p[n].requires_grad_(True) for n in ("a_in", "b_in", "a_out", "b_out")}

    def project(v, w, a, b):
        out = v @ w.t()
        for r in range(a.shape[0]):
            mine = (index == r).float()[:, None]
            out = out + mine * ((v @ a[r].t()) @ b[r].t()) * p["scale"][r]
        return out

    gate, value = project(x, p["w_in"], p["a_in"], p["b_in"]).chunk(2, 1)
    h = project(torch.nn.functional.silu(gate) * value, p["w_out"], p["a_out"], p["b_out"])
    loss = torch.nn.functional.cross_entropy(h @ p["head"].t(), target, reduction="none", ignore_index=-100)
    loss.backward(grad)
    return loss.detach(), {"x": x.grad, **{n: t.grad for n, t in leaves.items()}}


def main(tokens=4096, adapters=4, rank=16, width=2048, inner=4096, words=32768, seed=0, repeat=10):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda size, *s: (torch.randn(*s, generator=g, device="cuda") * size).bfloat16()  # noqa: E731
    p = {"w_in": normal(width ** -0.5, 2 * inner, width), "w_out": normal(inner ** -0.5, width, inner),
         "a_in": normal(width ** -0.5, adapters, rank, width), "b_in": normal(rank ** -0.5, adapters, 2 * inner, rank),
         "a_out": normal(inner ** -0.5, adapters, rank, inner), "b_out": normal(rank ** -0.5, adapters, width, rank),
         "scale": torch.ones(adapters, device="cuda"), "head": normal(width ** -0.5, words, width)}
    x = normal(1.0, tokens, width)
    # one request after the other, the last without an adapter; prompts do not count
    index = (torch.arange(tokens, device="cuda") * (adapters + 1) // tokens).to(torch.int32)
    target = torch.randint(0, words, (tokens,), generator=g, device="cuda")
    target[::5] = -100
    grad = torch.full((tokens,), 1.0 / tokens, device="cuda")

    def step():
        loss, saved = forward(x, p, index, target)
        return loss, backward(saved, grad)

    loss, grads = step()
    want_loss, want = plain(x, p, index, target, grad)
    off = {n: float((grads[n].float() - want[n]).norm() / want[n].norm()) for n in grads}
    off["loss"] = float((loss - want_loss).norm() / want_loss.norm())
    torch.cuda.synchronize()
    start, end = torch.cuda.Event(True), torch.cuda.Event(True)
    start.record()
    for _ in range(repeat):
        step()
    end.record()
    torch.cuda.synchronize()
    ms = start.elapsed_time(end) / max(repeat, 1)
    kept = tokens * (2 * inner * (1 + 4 / 128) + 2 * (width + 4 * rank))
    print(f"{tokens} tokens, {adapters} adapters of rank {rank}, {width} -> 2 x {inner} -> {width}, {words} words: "
          f"{ms:.3f} ms a step, {kept / 2 ** 20:.0f} MiB kept; off full precision by "
          + ", ".join(f"{n} {v:.4f}" for n, v in off.items()))
    return off


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("adapters", 4), ("rank", 16), ("width", 2048), ("inner", 4096),
                        ("words", 32768)):
        p.add_argument("--" + name, type=int, default=value)
    main(**vars(p.parse_args()))
