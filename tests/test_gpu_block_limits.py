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
