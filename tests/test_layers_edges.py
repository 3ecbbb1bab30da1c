"""CPU tests of include/gemm_layers.h at the edges of its sizes and arguments. No kernel is launched; a
call that would be made gives GEMM_ERR_DEVICE where there is no GPU, and is not made where there is one."""
import ctypes

import pytest
import torch

import dense_gemm_06_amd as dg

OK, INVALID, NULL, UNSUPPORTED, DEVICE = 0, 1, 2, 3, 4
TYPES = (dg.GEMM_F32, dg.GEMM_F16, dg.GEMM_BF16)
G = 1 << 40  # distance between the made-up addresses: nothing overlaps


def lib():
    return dg.library()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [0, 1, 16, 17, 20, 64, 65, 300, 5000])
def test_adapters_workspaces_of_empty_sizes(T, dtype):
    for N in (0, 1, 64):
        for K in (0, 1, 8, 64):
            for R, rank in ((0, 0), (0, 5), (1, 1), (3, 16), (2, 128)):
                assert lib().gemm_adapters_workspace(T, N, K, rank, dtype) >= 0
                assert lib().gemm_adapters_backward_workspace(T, N, K, R, rank, dtype) >= 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [0, 1, 65, 300])
def test_loss_workspaces_of_empty_sizes(T, dtype):
    for V in (0, 1, 7, 300):
        for K in (0, 1, 8, 64):
            assert lib().gemm_loss_workspace(T, V, K, dtype) >= 0
            for want in ((0, 0), (0, 1), (1, 0), (1, 1)):
                for piece in (0, 1, 1000):
                    assert lib().gemm_loss_backward_workspace(T, V, K, dtype, *want, piece) >= 0
