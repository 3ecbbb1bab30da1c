"""Plain definitions, in 64 bits on the CPU, of the operators around a layer's products, and the
error bounds of their tests. A sum of n products in fp32, in any order, is off by at most
n 2^-24 of the sum of their magnitudes; a rounding to a type by half a step (HALF)."""
from __future__ import annotations

import math

import torch

from block_util import HALF, TINY

F32 = 2.0 ** -24


def check(got, ref, bound, what):
    """|got - ref| <= bound everywhere (NaN where ref is NaN)."""
    got = got.cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= bound) & ~(got == ref) & ~(got.isnan() & ref.isnan())
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4], ref[bad][:4], bound[bad][:4])


def rounded(ref, dtype):
    """The last rounding to dtype."""
    return ref.abs() * HALF[dtype] * (1 + 2.0 ** -7) + TINY[dtype]


# ----------------------------------------------------------------------------- adapters
def masks(index, R):
    return [(index.cpu() == r).double()[:, None] for r in range(R)]


def kept_as(s, dtype):
    """The error of a number held as the sum of two of a 16-bit type."""
    if dtype == torch.float32:
        return s.abs() * F32
    return s.abs() * HALF[dtype] ** 2 * 2 + (2.0 ** -24 if dtype == torch.float16 else 2.0 ** -133)


def adapters(x, w, a, b, index, scale):
    """(y, u) with their bounds."""
    dt = x.dtype
    x, w, a, b = (t.cpu().double() for t in (x, w, a, b))
    R, K, rank = a.shape[0], x.shape[1], a.shape[1]
    s = torch.ones(R, dtype=torch.float64) if scale is None else scale.cpu().double()
    y, size = x @ w.t(), (x.abs() @ w.abs().t())
    err = size * (K + rank + 4) * F32
    u, u_size = x.new_zeros(len(x), rank), x.new_zeros(len(x), rank)
    for r, m in enumerate(masks(index, R)):
        u, u_size = u + m * (x @ a[r].t()), u_size + m * (x.abs() @ a[r].abs().t())
    u_err = u_size * (K + 2) * F32
    for r, m in enumerate(masks(index, R)):
        v = m * u * s[r]
        y = y + v @ b[r].t()
        v_err = m * u_err * s[r].abs() + v.abs() * 2 * F32 + m * kept_as(v, dt)
        err = err + (v.abs() @ b[r].abs().t()) * (K + rank + 4) * F32 + v_err @ b[r].abs().t() * (1 + 2.0 ** -8)
    return y, err + rounded(y, dt) + err * HALF[dt], u, u_err + TINY[torch.float32]


def adapters_backward(grad, x, u, w, a, b, index, scale):
    """x_grad, a_grad, b_grad with their bounds, for the kernel's own u as input."""
    dt = x.dtype
    g, x, u, w, a, b = (t.cpu().double() for t in (grad, x, u, w, a, b))
    T, N = g.shape
    R, rank = a.shape[0], a.shape[1]
    s = torch.ones(R, dtype=torch.float64) if scale is None else scale.cpu().double()
    xg, err = g @ w, (g.abs() @ w.abs()) * (N + rank + 4) * F32
    ag, ag_err, bg, bg_err = [], [], [], []
    for r, m in enumerate(masks(index, R)):
        v, v_size = m * (g @ b[r]) * s[r], m * (g.abs() @ b[r].abs()) * s[r].abs()
        v_err = v_size * (N + 3) * F32
        held = v_err + m * kept_as(v, dt)
        xg = xg + v @ a[r]
        err = err + (v.abs() @ a[r].abs()) * (N + rank + 4) * F32 + held @ a[r].abs() * (1 + 2.0 ** -8)
        rows = int(m.sum())
        ag.append(v.t() @ x)
        ag_err.append(held.t() @ x.abs() * (1 + 2.0 ** -8) + (v.abs().t() @ x.abs()) * (rows + 4) * F32)
        um = m * u
        bg.append(g.t() @ um * s[r])
        u_held = m * kept_as(u, dt)
        bg_err.append(((g.abs().t() @ um.abs()) * (rows + 6) * F32 + g.abs().t() @ u_held * (1 + 2.0 ** -8)) * s[r].abs())
    stack = lambda parts, shape: torch.stack(parts) if parts else torch.zeros(shape, dtype=torch.float64)  # noqa: E731
    ag, bg = stack(ag, a.shape), stack(bg, b.shape)
    ag_err, bg_err = stack(ag_err, a.shape), stack(bg_err, b.shape)
    grow = 1 + HALF[dt]
    return (xg, err * grow + rounded(xg, dt)), (ag, ag_err * grow + rounded(ag, dt)), (bg, bg_err * grow + rounded(bg, dt))


# ----------------------------------------------------------------------------- loss
def loss(x, w, target):
    """(loss, lse) with their bounds, and the logits with theirs."""
    x, w, target = x.cpu().double(), w.cpu().double(), target.cpu()
    V, K = w.shape
    l, l_err = x @ w.t(), (x.abs() @ w.abs().t()) * (K + 1) * F32
    lse = torch.logsumexp(l, 1)
    top = l.amax(1) if V else torch.zeros(len(x))
    spread = (top - l.amin(1)) if V else torch.zeros(len(x))
    # each exponential's argument is rounded (log2(e) in fp32 too), the sum has V terms
    lse_err = l_err.amax(1) if V else torch.zeros(len(x), dtype=torch.float64)
    lse_err = lse_err + (V + 64 + 4 * spread) * F32 + 4 * F32 * (lse.abs() + top.abs())
    live = (target >= 0) & (target < V)
    at = torch.where(live, target, 0)[:, None]
    picked = l.gather(1, at)[:, 0] if V else torch.zeros(len(x), dtype=torch.float64)
    value = torch.where(live, lse - picked, 0.0)
    err = lse_err + (l_err.gather(1, at)[:, 0] if V else 0) + 2 * F32 * (lse.abs() + picked.abs())
    return value, err, lse, lse_err, l, l_err


def loss_backward(grad, x, w, target, lse):
    """(x_grad, w_grad) with their bounds, for the kernel's own lse as input."""
    dt = x.dtype
    g, given = grad.cpu().double(), lse.cpu().double()
    _, _, _, _, l, l_err = loss(x, w, target)
    x, w, target = x.cpu().double(), w.cpu().double(), target.cpu()
    V, T = w.shape[0], len(x)
    live = ((target >= 0) & (target < V)).double()
    hit = torch.nn.functional.one_hot(target.clamp(0, V - 1), V).double()
    p = torch.exp(l - given[:, None])
    scale = (g * live).abs()[:, None]
    d = (p - hit) * (g * live)[:, None]
    arg = (l - given[:, None]).abs()
    d_err = scale * (p * (torch.expm1(l_err) + (4 * arg + 8) * F32) + (p + hit) * 3 * F32)
    # an exponential, or a d, below the smallest normal number 2^-126 may count as zero: off by less than that
    d_err = d_err + (scale + 1) * (scale > 0) * 2.0 ** -126
    dx_err = dw_err = d_err
    if dt != torch.float32:
        # d is rounded. Rows of 8 and more: the target's -1 is left out of x's where p < 1/2 (p < 0.51 here:
        # the kernel's p decides) and added in fp32, and w's gets what the target's rounding took, rounded
        left_out = hit if x.shape[1] >= 8 else 0 * hit
        dx_err = dx_err + (torch.where((left_out > 0) & (p < 0.49), p, (p - hit).abs()) * scale) * HALF[dt] * 1.01
        dx_err = dx_err + left_out * ((p >= 0.49) & (p < 0.51)) * scale * HALF[dt] * 0.03
        dw_err = dw_err + d.abs() * torch.where(left_out > 0, HALF[dt] ** 2, HALF[dt]) * 1.01
        if dt == torch.float16:
            # held times a power of two that brings the largest |g| to 2^13 .. 2^14
            low = 2.0 ** -25 * 2.0 ** (math.frexp(float(g.abs().max()))[1] - 13) * (scale > 0)
            dx_err, dw_err = dx_err + low, dw_err + low
    grow = 1 + HALF[dt]
    xg, wg = d @ w, d.t() @ x
    xg_err = dx_err @ w.abs() * 1.01 + ((d.abs() + 2 * hit * scale) @ w.abs()) * (V + 40) * F32
    wg_err = dw_err.t() @ x.abs() * 1.01 + (d.abs().t() @ x.abs()) * (T + 4) * F32
    return (xg, xg_err * grow + rounded(xg, dt)), (wg, wg_err * grow + rounded(wg, dt))


# ----------------------------------------------------------------------------- activations
def act(v, kind):
    """f, f' and bounds of their fp32 computation."""
    if kind == "relu":
        f, d = torch.where(v > 0, v, 0.0), (v > 0).double()
        return f, d, torch.zeros_like(v), torch.zeros_like(v)
    w2 = v if kind == "silu" else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
    dw2 = torch.ones_like(v) if kind == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * v * v)
    s, r = torch.sigmoid(w2), torch.sigmoid(-w2)
    # e^-w2: w2 is off by 4 roundings, the exponential and the reciprocal by a few steps; s turns
    # e's relative error into r times it
    rel = (12 + 4 * w2.abs() * r) * F32
    f, d = v * s, s + v * s * r * dw2
    part = (v * s * r * dw2).abs()
    # past e = 2^100 .. 2^128 the products leave fp32's normal numbers
    tiny = 2.0 ** -96 * (1 + v.abs())
    return f, d, f.abs() * rel + tiny, s * rel + part * ((24 + 8 * w2.abs()) * F32) + tiny * dw2


def activation(z, kind, gated):
    dt = z.dtype
    z = z.cpu().double()
    F = z.shape[1] // 2 if gated else z.shape[1]
    f, _, f_err, _ = act(z[:, :F], kind)
    if gated:
        f, f_err = f * z[:, F:], f_err * z[:, F:].abs() * 1.01 + (f * z[:, F:]).abs() * F32
    return f, f_err * 1.01 + rounded(f, dt) + 2.0 ** -149


def activation_backward(grad, z, kind, gated):
    """z_grad and y with their bounds; z: the codes' values in 64 bits, which the kernel rounds to fp32."""
    dt = grad.dtype
    g = grad.cpu().double()
    F = g.shape[1]
    v = z[:, :F]
    f, d, f_err, d_err = act(v, kind)
    if kind != "relu":  # the values' own rounding
        w2 = v.abs() if kind == "silu" else 1.6 * (v.abs() + 0.045 * v.abs() ** 3)
        f_err, d_err = f_err + f.abs() * (2 + 3 * w2) * F32, d_err * 1.5 + (4 + 3 * w2) * F32 * d.abs().clamp(min=0.0)
    else:
        f_err = f_err + f.abs() * F32
    if not gated:
        zg, zg_err, y, y_err = g * d, g.abs() * d_err * 1.01 + (g * d).abs() * F32, f, f_err
    else:
        u = z[:, F:]
        z1, z2 = g * d * u, g * f
        zg = torch.cat([z1, z2], 1)
        zg_err = torch.cat([(g * u).abs() * d_err * 1.01 + 4 * F32 * z1.abs(), g.abs() * f_err * 1.01 + F32 * z2.abs()], 1)
        y, y_err = f * u, f_err * u.abs() * 1.01 + (f * u).abs() * 3 * F32
    return (zg, zg_err * 1.01 + rounded(zg, dt) + 2.0 ** -149), (y, y_err * 1.01 + rounded(y, dt) + 2.0 ** -149)
