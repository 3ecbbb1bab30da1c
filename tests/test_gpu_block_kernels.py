"""GPU tests of every kernel of the block-scaled products (tests/block_shapes.py), with every pair
of types and both kinds of scales of B, against 64-bit products on the CPU. For every C: sums in
fp32, one rounding to its type."""
import pytest
import torch

import dense_gemm_06_amd as dg
from block_shapes import EXPERTS, GRADIENT, PLAIN, SHAPES
from block_util import BLOCK, HALF, TINY, blocks, codes, values

pytestmark = pytest.mark.gpu

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def check(got, a, b, dtype, what):
    """128 exact products summed in fp32 in any order, two factors, the sum over blocks in fp32, one rounding."""
    K = a.shape[1]
    ref, size = a @ b.t(), a.abs() @ b.abs().t()
    bound = size * (BLOCK + blocks(K) + 3) * 2.0 ** -24 + ref.abs() * HALF[dtype] * (1 + 2.0 ** -9) + TINY[dtype]
    bad = ~((got.cpu().double() - ref).abs() <= bound)
    assert got.dtype == dtype and not bad.any(), (what, int(bad.sum()))


def laid(q, turned, odd):
    """Codes on the GPU: rows contiguous or adjacent, at multiples of 16 bytes or at odd ones."""
    q = q.cuda()
    if turned:
        q = q.transpose(-1, -2).contiguous()
    if odd:
        wide = torch.zeros(*q.shape[:-1], q.shape[-1] + 3, dtype=torch.uint8, device="cuda")
        wide[..., 1:1 + q.shape[-1]].copy_(q.view(torch.uint8))
        q = wide.view(q.dtype)[..., 1:1 + q.shape[-1]]
    return q.transpose(-1, -2) if turned else q


def tensor(c, block_rows, turned, odd):
    s = c[1]
    return dg.BlockTensor(laid(c[0], turned, odd), s.transpose(-1, -2).contiguous().transpose(-1, -2).cuda(), block_rows)


@pytest.mark.parametrize("shape", SHAPES, ids=repr)
def test_kernel(shape):
    g = gen(sum(shape.sizes))
    pairs = ((E4, E4, BF16), (E4, E5, F32), (E5, E4, F16), (E5, E5, BF16), (E4, E4, F32), (E4, E4, F16))
    ta, tb, odd = "a" in shape.turn, "b" in shape.turn, shape.odd
    if shape.mode == PLAIN:
        M, N, K = shape.sizes
        for i, (qa, qb, out) in enumerate(pairs if M * N < 1 << 20 else pairs[:2]):
            for rows in shape.b_rows:
                a, b = codes(g, M, K, qa, 1), codes(g, N, K, qb, rows)
                c = dg.gemm_block_product_tensors(tensor(a, 1, ta, odd), tensor(b, rows, tb, odd), out)
                check(c, values(*a, 1), values(*b, rows), out, (qa, qb, out, rows))
        return
    T, k, E, x, y = shape.sizes
    index = torch.topk(torch.randn(T, E, generator=g) + torch.randn(1, E, generator=g), k, dim=1).indices.to(torch.int32)
    index[index == E - 2] = -1                           # an expert without rows, and rows without an expert
    plan = dg.gemm_experts_dispatch_tensors(index.cuda(), E, shape.align)
    off, cnt, rows = plan.offsets.tolist(), plan.counts.tolist(), plan.rows.cpu().long()
    P = len(rows)
    for qa, qb, out in pairs[:3]:
        if shape.mode == EXPERTS:
            for scale_rows in shape.b_rows:
                b = codes(g, x, y, qb, scale_rows, batch=E)
                live = torch.zeros(P, dtype=torch.bool)
                for gather in (True, False):
                    a = codes(g, T if gather else P, y, qa, 1)
                    A, B = tensor(a, 1, ta, odd), tensor(b, scale_rows, tb, odd)
                    c = dg.gemm_experts_product_tensors(A, B, plan, out, gather)
                    va = values(*a, 1)
                    for e in range(E):
                        at = slice(off[e], off[e] + cnt[e])
                        live[at] = True
                        if cnt[e]:
                            check(c[at], va[rows[at]] if gather else va[at], values(b[0][e], b[1][e], scale_rows), out, (qa, qb, out, e))
                    assert (c.cpu()[~live] == 0).all()
            continue
        for scale_rows in shape.b_rows:
            a, b = codes(g, x, P, qa, 1), codes(g, y, P, qb, scale_rows)
            c = dg.gemm_experts_gradient_tensors(tensor(a, 1, ta, odd), tensor(b, scale_rows, tb, odd), plan, out)
            va, vb = values(*a, 1), values(*b, scale_rows)
            for e in range(E):
                check(c[e], va[:, off[e]:off[e + 1]], vb[:, off[e]:off[e + 1]], out, (qa, qb, out, e))


def test_transposed_codes_of_the_quantizer():
    """The gradient's operands as a training step has them: rows contiguous, from the quantizer's transposed form."""
    g = gen(5)
    T, k, E, M, N = 900, 2, 3, 300, 200
    index = torch.topk(torch.randn(T, E, generator=g), k, dim=1).indices.to(torch.int32)
    plan = dg.gemm_experts_dispatch_tensors(index.cuda(), E, BLOCK)
    x, y = torch.randn(T, M, generator=g).to(BF16).cuda(), torch.randn(T, N, generator=g).to(BF16).cuda()
    _, a = dg.gemm_block_quantize_tensors(x, E5, natural=False, transposed=True, rows=plan.rows)
    _, b = dg.gemm_block_quantize_tensors(y, E4, natural=False, transposed=True, rows=plan.rows)
    assert a.data.stride(-1) == 1 and b.data.stride(-1) == 1
    c = dg.gemm_experts_gradient_tensors(a, b, plan)
    off = plan.offsets.tolist()
    for e in range(E):
        check(c[e], values(a.data, a.scale, 1)[:, off[e]:off[e + 1]], values(b.data, b.scale, 1)[:, off[e]:off[e + 1]], F32, e)
