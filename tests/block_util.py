"""Plain definitions, in 64 bits on the CPU, of the block-scaled and experts' operators, and
the error bounds of their tests (a rounding to a type is off by at most half a step)."""
from __future__ import annotations

import math

import torch

BLOCK = 128
QMAX = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}


def blocks(n):
    return -(-n // BLOCK)


def quantize(x, dtype, block_rows):
    """The definition with its fp32 roundings: (codes, scales) of a 2-D tensor on the CPU."""
    x = x.float()
    R, K = x.shape
    pad = torch.zeros(-(-R // block_rows) * block_rows, blocks(K) * BLOCK)
    pad[:R, :K] = x
    amax = pad.abs().reshape(-1, block_rows, blocks(K), BLOCK).amax(dim=(1, 3)).clamp(min=2.0 ** -100)
    top = torch.full_like(amax, QMAX[dtype])
    inv = (top / amax).repeat_interleave(block_rows, 0)[:R].repeat_interleave(BLOCK, 1)[:, :K]
    return (x * inv).to(dtype), amax / top


def values(data, scale, block_rows):
    """The numbers that codes and scales stand for, in 64 bits on the CPU."""
    R, K = data.shape[-2:]
    s = scale.cpu().double().repeat_interleave(block_rows, -2)[..., :R, :].repeat_interleave(BLOCK, -1)[..., :K]
    return data.cpu().float().double() * s


def product_bound(a, b, ref, size, dtype):
    """|error| of a product: 128 exact products summed in fp32 in any order, the two scales' product and
    the sum over blocks in fp32, one rounding to the output's type. size: the sums of |a||b|. For outputs
    of 16 bits the products of 8 neighbouring k are first cut to multiples of 2^-13 of the power of two
    under the largest: less than 2^-13 of the largest for each of the 7 others."""
    K = a.shape[1]
    bound = size * (BLOCK + blocks(K) + 3) * 2.0 ** -24 + ref.abs() * HALF[dtype] * (1 + 2.0 ** -9) + TINY[dtype]
    if dtype != torch.float32:
        top = lambda x: torch.nn.functional.pad(x.abs(), (0, -K % 8)).reshape(x.shape[0], -1, 8).amax(2)  # noqa: E731
        bound = bound + top(a) @ top(b).t() * (7 * 2.0 ** -13) * (1 + 2.0 ** -9)
    return bound


def check_product(got, a, b, dtype, what=""):
    """got against a b^T for 64-bit a (M, K), b (N, K)."""
    ref, size = a @ b.t(), a.abs() @ b.abs().t()
    err, bound = (got.cpu().double() - ref).abs(), product_bound(a, b, ref, size, dtype)
    assert got.dtype == dtype and tuple(got.shape) == tuple(ref.shape)
    bad = ~(err <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((err / bound.clamp(min=1e-300)).max()))


def codes(g, rows, cols, dtype, block_rows, batch=None, spread=1.0):
    """Seeded codes and scales on the CPU: (data, scale) of normal values whose columns differ in size."""
    lead = () if batch is None else (batch,)
    x = torch.randn(*lead, rows, cols, generator=g) * torch.exp(spread * torch.randn(*lead, 1, cols, generator=g))
    flat = x.reshape(-1, cols) if batch is None else x
    if batch is None:
        return quantize(flat, dtype, block_rows)
    parts = [quantize(m, dtype, block_rows) for m in x]
    return torch.stack([p[0].view(torch.uint8) for p in parts]).view(dtype), torch.stack([p[1] for p in parts])


def scores(logits, kind):
    x = logits.double()
    if kind == "sigmoid":
        return torch.sigmoid(x)
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def route(logits, bias, k, kind, groups, top_groups, group_top, renorm, factor):
    """(index, weight) by explicit loops over a token's experts, in 64 bits."""
    s = scores(logits, kind)
    c = s if bias is None else s + bias.double()
    T, E = s.shape
    index, weight = torch.empty(T, k, dtype=torch.int32), torch.empty(T, k, dtype=torch.float64)
    for t in range(T):
        row = c[t].tolist()
        allowed = range(E)
        if groups > 1:
            per = E // groups
            best = [sum(sorted(row[g * per:(g + 1) * per], reverse=True)[:group_top]) for g in range(groups)]
            kept = sorted(range(groups), key=lambda g: (-best[g], g))[:top_groups]
            allowed = [e for g in sorted(kept) for e in range(g * per, (g + 1) * per)]
        pick = sorted(allowed, key=lambda e: (-row[e], e))[:k]
        w = s[t, pick]
        if renorm:
            w = w / w.sum()
        index[t], weight[t] = torch.tensor(pick, dtype=torch.int32), w * factor
    return index, weight


def dispatch(index, E, align, P):
    """offsets, counts, rows, position by walking the pairs in order."""
    T, k = index.shape
    lists = [[] for _ in range(E)]
    for i, e in enumerate(index.reshape(-1).tolist()):
        if 0 <= e < E:
            lists[e].append(i)
    offsets, rows, position = [0], [-1] * P, [-1] * (T * k)
    for e in range(E):
        at = offsets[-1]
        for r, i in enumerate(lists[e]):
            rows[at + r], position[i] = i // k, at + r
        offsets.append(at + math.ceil(len(lists[e]) / align) * align)
    as_i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return as_i32(offsets), as_i32([len(x) for x in lists]), as_i32(rows), as_i32(position).reshape(T, k)
