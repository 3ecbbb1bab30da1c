"""GPU tests of the block-scaled and experts' operators at sizes next to 2^31."""
import pytest
import torch

import dense_gemm_06_amd as dg

pytestmark = pytest.mark.gpu

E4 = torch.float8_e4m3fn
F32, BF16 = torch.float32, torch.bfloat16


def test_product_of_the_longest_rows():
    """K = 2^31 - 1: whole blocks and a cut one, numbers in the first, in between and in the last."""
    K = 2 ** 31 - 1
    one = torch.zeros(1, K, dtype=torch.uint8, device="cuda")
    at = [0, 127, 2 ** 20 + 5, 2 ** 30, K - 128, K - 127, K - 1]
    one[0, at] = 0x38                                    # 1.0
    scale = torch.ones(1, 1, device="cuda").expand(1, 2 ** 24)
    a = dg.BlockTensor(one.view(E4), scale, 1)
    for out in (F32, BF16):
        assert dg.gemm_block_product_tensors(a, a, out).item() == len(at)


def test_combine_of_the_longest_rows():
    """2^31 - 1 columns: the last whole pass of a workgroup ends within one pass of 2^31."""
    N = 2 ** 31 - 1
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    plan = dg.ExpertPlan(i32(0, 1), i32(1), i32(0), i32(0).reshape(1, 1))
    at = [0, 2047, 2048, 2 ** 30, N - 2048, N - 2047, N - 1]
    y = torch.zeros(1, N, dtype=BF16, device="cuda")
    y[0, at] = 3.0
    weight = torch.full((1, 1), 0.5, device="cuda")
    out = dg.gemm_experts_combine_tensors(y, plan, weight)
    assert out[0, at].tolist() == [1.5] * len(at) and int(torch.count_nonzero(out[0])) == len(at)
    y_grad, weight_grad = dg.gemm_experts_combine_backward_tensors(y, plan, weight, out)
    assert y_grad[0, at].tolist() == [0.75] * len(at) and int(torch.count_nonzero(y_grad[0])) == len(at)
    assert weight_grad.item() == 4.5 * len(at)


@pytest.mark.parametrize("T,N", [(8, 64), (300, 200)])
def test_offsets_that_overlap_stay_inside(T, N):
    """A plan whose offsets go back and forth: whatever comes out, nothing beside C is written."""
    P, E = 2 * T, 40
    g = torch.Generator().manual_seed(T)
    offsets = torch.tensor([0, P] * (E // 2) + [P], dtype=torch.int32)
    offsets[5], offsets[7], offsets[9] = -3, 2 ** 31 - 1, -2 ** 31
    rows = torch.randint(-2, T + 2, (P,), generator=g).to(torch.int32)
    counts = torch.full((E,), P + 9, dtype=torch.int32)
    plan = dg.ExpertPlan(offsets.cuda(), counts.cuda(), rows.cuda(), torch.zeros(T, 2, dtype=torch.int32, device="cuda"))
    one = lambda *s: torch.full(s, 0x38, dtype=torch.uint8, device="cuda").view(E4)  # noqa: E731
    a = dg.BlockTensor(one(T, 128), torch.ones(T, 1, device="cuda"), 1)
    b = dg.BlockTensor(one(E, N, 128), torch.ones(E, 2 if N > 128 else 1, 1, device="cuda"), 128)
    for out in (F32, BF16):
        wide = torch.full((P + 512, N + 64), 7.0, dtype=out, device="cuda")
        A, B, p = dg.experts._block(a, "a"), dg.experts._block(b, "b", 3), dg.experts._plan(plan)
        dg.experts._call("gemm_experts_product", 0, A, B, p, 1, wide[256].data_ptr(), N + 64, dg.experts._WIDE[out])
        c = wide[256:256 + P, :N]
        live = torch.tensor([0 <= r < T for r in rows.tolist()])
        assert set(c[live.cuda()].unique().tolist()) <= {0.0, 128.0} and (c[~live.cuda()] == 0).all()
        wide[256:256 + P, :N] = 7.0
        assert (wide == 7.0).all()


def test_rows_without_experts():
    """A plan of no experts: its rows are padding."""
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for P, N in ((5, 40), (300, 200)):
        plan = dg.ExpertPlan(i32(0), i32(), i32(*[-1] * P), i32(-1).reshape(1, 1))
        a = dg.BlockTensor(torch.ones(1, 128, device="cuda").to(E4), torch.ones(1, 1, device="cuda"), 1)
        b = dg.BlockTensor(torch.empty(0, N, 128, device="cuda").to(E4), torch.empty(0, -(-N // 128), 1, device="cuda"), 128)
        for out in (F32, BF16):
            c = dg.gemm_experts_product_tensors(a, b, plan, out)
            assert c.shape == (P, N) and (c == 0).all()
