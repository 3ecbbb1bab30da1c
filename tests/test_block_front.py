"""CPU tests of how the torch front passes on the layouts of block-scaled matrices."""
import pytest
import torch

import dense_gemm_06_amd as dg
from dense_gemm_06_amd import experts

E4 = torch.float8_e4m3fn


def codes(*shape):
    return torch.zeros(*shape, dtype=torch.uint8).view(E4)


def passed(data, block_rows=1):
    experts._use_torch()
    R, K = data.shape[-2:]
    scale = torch.ones(*data.shape[:-2], -(-R // block_rows), -(-K // 128))
    return experts._block(dg.BlockTensor(data, scale, block_rows), "a", data.dim())


@pytest.mark.parametrize("data,ld,op", [
    (codes(5, 300), 300, 0), (codes(5, 320)[:, :300], 320, 0), (codes(1, 300), 300, 0), (codes(7, 1), 1, 0),
    (codes(300, 5).t(), 5, 1), (codes(300, 8).t()[:5], 8, 1), (codes(300, 8).t()[:1], 8, 1), (codes(300, 1).t(), 300, 0),
    (codes(2, 300, 8).transpose(1, 2)[:, 2:3], 8, 1), (codes(1, 1), 1, 0)], ids=lambda x: "x".join(map(str, x.shape)) if torch.is_tensor(x) else str(x))
def test_either_dimension_contiguous(data, ld, op):
    """Rows that are contiguous, or columns; a matrix of one row lies both ways."""
    m = passed(data)
    assert (m.rows, m.cols, m.ld, m.op) == (data.shape[-2], data.shape[-1], ld, op) and m.data == data.data_ptr()
    # the library's own reading of these fields finds every element
    step = data.stride(-1) if data.shape[-1] > 1 else 1
    assert (m.ld if m.op else 1) == step or data.shape[-1] == 1


def test_no_contiguous_dimension_is_refused():
    with pytest.raises(ValueError, match="unit stride"):
        passed(codes(10, 600)[:, ::2])
    with pytest.raises(ValueError, match="overlap"):
        passed(codes(700).as_strided((5, 300), (1, 2)))


@pytest.mark.gpu
@pytest.mark.parametrize("N,K", [(1, 300), (200, 256)])
def test_one_sliced_row(N, K):
    """One row of a wider matrix stored the other way round, times whole and single rows."""
    g = torch.Generator().manual_seed(N)
    a = torch.randint(-4, 5, (K, 6), generator=g).float()
    b = torch.randint(-4, 5, (N, K), generator=g).float()
    A = dg.BlockTensor(a.to(E4).cuda().t()[2:3], torch.ones(1, -(-K // 128), device="cuda"), 1)
    B = dg.BlockTensor(b.to(E4).cuda(), torch.ones(N, -(-K // 128), device="cuda"), 1)
    want = (a.t()[2:3].double() @ b.double().t()).float()
    assert torch.equal(dg.gemm_block_product_tensors(A, B, torch.float32).cpu(), want)
    assert torch.equal(dg.gemm_block_product_tensors(B, A, torch.float32).cpu(), want.t())
