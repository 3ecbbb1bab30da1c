"""GPU tests of block-scaled products whose two scales multiply to no normal fp32 number although
the scaled sums are."""
import pytest
import torch

import dense_gemm_06_amd as dg
from block_util import BLOCK, HALF, TINY, blocks, values

pytestmark = pytest.mark.gpu

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def numbers(g, kind, rows, cols, block_rows, batch=()):
    """Codes and scales of one operand. tiny: usual codes, scales of about 2^-70, so that two multiply to a
    subnormal number or to zero; huge: the smallest codes, scales of about 2^66, whose product is infinite; zero:
    codes of zero, with such scales."""
    shape = (*batch, rows, cols)
    if kind == "tiny":
        q, at = torch.randint(-448, 449, shape, generator=g).float().to(E4), -70
    else:
        q, at = (torch.randint(-2, 3, shape, generator=g).float() * (2.0 ** -9 if kind == "huge" else 0.0)).to(E4), 66
    s = (1 + torch.rand(*batch, -(-rows // block_rows), blocks(cols), generator=g)) * 2.0 ** at
    return q, s


def check(got, a, b, dtype):
    """The bound of fp32 sums: 128 exact products, two factors, the sum over blocks (whose roundings of numbers
    below the normal ones are at most half of 2^-149 each), one rounding to C's type."""
    K = a.shape[1]
    ref, size = a @ b.t(), a.abs() @ b.abs().t()
    bound = size * (BLOCK + blocks(K) + 3) * 2.0 ** -24 + blocks(K) * 2.0 ** -149 + ref.abs() * HALF[dtype] * (1 + 2.0 ** -9) + TINY[dtype]
    assert ((got.cpu().double() - ref).abs() <= bound).all()


def block(q, s, block_rows, ld=0, flip=False):
    q = q.cuda()
    if ld:
        wide = torch.zeros(q.shape[0], q.shape[1] + ld, device="cuda").to(E4)
        wide[:, 1:1 + q.shape[1]].view(torch.uint8).copy_(q.view(torch.uint8))
        q = wide[:, 1:1 + q.shape[1]]
    if flip:
        q = q.t().contiguous().t()
    return dg.BlockTensor(q, s.cuda(), block_rows)


FORMS = [(3, 80, 512, {}), (50, 64, 272, {}), (20, 70, 130, {"ld": 3}), (140, 300, 400, {}), (300, 200, 2064, {}),
         (200, 140, 300, {"ld": 5}), (140, 272, 384, {"flip": True})]


@pytest.mark.parametrize("M,N,K,how", FORMS, ids=str)
@pytest.mark.parametrize("b_rows", [1, BLOCK])
@pytest.mark.parametrize("kind", ["tiny", "huge", "zero"])
def test_product_of_scales_out_of_range(M, N, K, how, b_rows, kind):
    g = gen(M + N)
    a, b = numbers(g, kind, M, K, 1), numbers(g, kind, N, K, b_rows)
    A = block(*a, 1, how.get("ld", 0))
    B = block(*b, b_rows, how.get("ld", 0), how.get("flip", False))
    for out in (F32, BF16):
        check(dg.gemm_block_product_tensors(A, B, out), values(*a, 1), values(*b, b_rows), out)


@pytest.mark.parametrize("T,k,E,N,K", [(5, 2, 4, 80, 256), (200, 2, 4, 200, 272)])
@pytest.mark.parametrize("kind", ["tiny", "huge", "zero"])
def test_experts_scales_out_of_range(T, k, E, N, K, kind):
    g = gen(T)
    index = torch.topk(torch.randn(T, E, generator=g), k, dim=1).indices.to(torch.int32)
    plan = dg.gemm_experts_dispatch_tensors(index.cuda(), E, 128)
    a, b = numbers(g, kind, T, K, 1), numbers(g, kind, N, K, BLOCK, (E,))
    off, cnt, rows = plan.offsets.tolist(), plan.counts.tolist(), plan.rows.cpu().long()
    for out in (F32, BF16):
        c = dg.gemm_experts_product_tensors(block(*a, 1), block(*b, BLOCK), plan, out)
        for e in range(E):
            at = slice(off[e], off[e] + cnt[e])
            check(c[at], values(*a, 1)[rows[at]], values(b[0][e], b[1][e], BLOCK), out)


def test_one_block_out_of_range_beside_others():
    """Blocks in and out of the normal range in one sum, and scales of zero, infinity and NaN, which count as they
    are: a row with an infinite scale is infinite or NaN, the others are not touched."""
    g = gen(1)
    M, N, K = 140, 200, 640
    a, b = numbers(g, "tiny", M, K, 1), numbers(g, "tiny", N, K, BLOCK)
    a[1][:, 1] *= 2.0 ** 70
    b[1][:, 1] *= 2.0 ** 60
    a[1][:, 2] = 0.0
    a[1][3, 3], a[1][77, 0] = float("inf"), float("nan")
    c = dg.gemm_block_product_tensors(block(*a, 1), block(*b, BLOCK), F32)
    bad = torch.zeros(M, dtype=torch.bool)
    bad[3] = bad[77] = True
    assert not torch.isfinite(c[bad.cuda()]).any()
    check(c[(~bad).cuda()], values(*a, 1)[~bad], values(*b, BLOCK), F32)
