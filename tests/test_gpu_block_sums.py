"""GPU tests of the precision in which block-scaled products are summed: whole numbers whose
large products cancel within every 8 neighbouring k, so that each partial sum is exact in fp32
(below 2^24) and every C has one right value, whatever its type."""
import pytest
import torch

import dense_gemm_06_amd as dg
from block_util import BLOCK, blocks

pytestmark = pytest.mark.gpu

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def cancelling(g, M, N, K):
    """(a, b), whole numbers in 8 bits: in each 8 k, 448 * 448 and -448 * 448 at two of them and products of
    -1, 0 and 1 at the others."""
    a, b = (torch.randint(-1, 2, (n, K), generator=g).float() for n in (M, N))
    lanes = torch.stack([torch.randperm(8, generator=g)[:2] for _ in range(K // 8)]) + 8 * torch.arange(K // 8)[:, None]
    a[:, lanes[:, 0]], a[:, lanes[:, 1]] = 448.0, 448.0
    b[:, lanes[:, 0]], b[:, lanes[:, 1]] = 448.0, -448.0
    return a, b


def operand(x, flip=False, ld=0, block_rows=1):
    """x's codes with scales of one; flip: stored with the rows adjacent; ld: within rows of so many more."""
    q = x.to(E4)
    assert torch.equal(q.float(), x)
    if ld:
        wide = torch.zeros(*x.shape[:-1], x.shape[-1] + ld, device="cuda").to(E4)
        view = wide[..., 1:1 + x.shape[-1]]
        view.view(torch.uint8).copy_(q.view(torch.uint8))
        q = view
    else:
        q = q.cuda()
    if flip:
        q = q.transpose(-1, -2).contiguous().transpose(-1, -2)
    scale = torch.ones(*x.shape[:-2], -(-x.shape[-2] // block_rows), blocks(x.shape[-1]), device="cuda")
    return dg.BlockTensor(q, scale, block_rows)


FORMS = [(1, 128, 128, {}), (16, 100, 640, {}), (30, 64, 272, {}), (64, 80, 4096, {}), (9, 70, 130, {"ld": 3}),
         (100, 200, 400, {}), (257, 130, 512, {}), (130, 140, 300, {"ld": 7}), (90, 48, 256, {"fb": True}),
         (140, 272, 256, {"fa": True}), (96, 160, 130, {"fa": True, "fb": True}), (300, 300, 2048, {}),
         (2000, 3300, 1040, {}), (2000, 3280, 1040, {"fb": True})]


@pytest.mark.parametrize("M,N,K,how", FORMS, ids=str)
@pytest.mark.parametrize("b_rows", [1, BLOCK])
def test_products_that_cancel(M, N, K, how, b_rows):
    a, b = cancelling(gen(M + N + K), M, N, K)
    want = a.double() @ b.double().t()
    A = operand(a, how.get("fa", False), how.get("ld", 0))
    B = operand(b, how.get("fb", False), how.get("ld", 0), b_rows)
    for out in (BF16, F16, F32):
        assert torch.equal(dg.gemm_block_product_tensors(A, B, out).cpu(), want.to(out)), out


@pytest.mark.parametrize("T,k,E,N,K,align", [(16, 4, 64, 528, 256, 1), (7, 2, 4, 100, 400, 128), (200, 2, 8, 256, 272, 1),
                                             (333, 6, 10, 264, 400, 128)])
def test_experts_that_cancel(T, k, E, N, K, align):
    g = gen(T)
    index = torch.topk(torch.randn(T, E, generator=g), k, dim=1).indices.to(torch.int32)
    plan = dg.gemm_experts_dispatch_tensors(index.cuda(), E, align)
    a, b = cancelling(g, T, N, K)
    b = torch.stack([torch.where(b.abs() > 1, b, b.roll(e, 0)) for e in range(E)])
    off, cnt, rows = plan.offsets.tolist(), plan.counts.tolist(), plan.rows.cpu().long()
    want = torch.zeros(len(rows), N, dtype=torch.float64)
    for e in range(E):
        at = slice(off[e], off[e] + cnt[e])
        want[at] = a[rows[at]].double() @ b[e].double().t()
    A, B = operand(a), operand(b, block_rows=BLOCK)
    for out in (BF16, F16, F32):
        assert torch.equal(dg.gemm_experts_product_tensors(A, B, plan, out).cpu(), want.to(out)), out


@pytest.mark.parametrize("M,N,P", [(48, 130, 384), (130, 200, 512)])
@pytest.mark.parametrize("flip", [False, True])
def test_gradients_that_cancel(M, N, P, flip):
    a, b = cancelling(gen(M), M, N, P)
    ends = [0, 128, 128, P]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    plan = dg.ExpertPlan(i32(ends), i32([128, 0, P - 128]), i32([0] * P), i32([[0]]), BLOCK)
    for out in (BF16, F16, F32):
        c = dg.gemm_experts_gradient_tensors(operand(a), operand(b, flip), plan, out).cpu()
        for e in range(3):
            want = a[:, ends[e]:ends[e + 1]].double() @ b[:, ends[e]:ends[e + 1]].double().t()
            assert torch.equal(c[e], want.to(out)), (e, out)


def test_terms_just_under_a_cut():
    """One product of 448 * 448 in each 8 k and seven of about 2^-13 of it, all of one sign: their sum counts."""
    for M in (5, 140):
        a, b = torch.full((M, 256), 4.5), torch.full((144, 256), 5.0)
        a[:, ::8], b[:, ::8] = 448.0, 448.0
        want = a.double() @ b.double().t()
        assert want.max() < 2 ** 24
        assert torch.equal(dg.gemm_block_product_tensors(operand(a), operand(b), F32).cpu().double(), want)
        half = dg.BlockTensor(operand(a).data, torch.full((M, 2), 2.0 ** -9, device="cuda"), 1)  # within fp16's range
        for out in (BF16, F16):
            assert torch.equal(dg.gemm_block_product_tensors(half, operand(b), out).cpu(), (want * 2.0 ** -9).to(out)), out
