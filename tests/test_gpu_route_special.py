"""GPU tests of routing with infinite and NaN choice values in groups."""
import pytest
import torch

import dense_gemm_06_amd as dg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,groups", [(64, 4), (60, 5), (256, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_excluded_experts_of_the_kept_groups(E, groups, score):
    """Fewer live experts in the kept group than choices: its excluded ones (bias of -inf) come next, by index, and
    none of another group."""
    per = E // groups
    bias = torch.full((E,), -float("inf"))
    bias[2 * per + 4] = 0.0
    for group_top in (1, 2):
        r = dg.router(3, score, groups=groups, top_groups=1, group_top=group_top)
        index, _ = dg.gemm_experts_route_tensors(torch.zeros(2, E).cuda(), r, bias.cuda())
        want = [2 * per + 4, 2 * per, 2 * per + 1] if group_top == 1 else [0, 1, 2]   # sums with -inf: all groups tie
        assert index.tolist() == [want, want]
