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


@pytest.mark.parametrize("E,groups", [(64, 4), (60, 5), (256, 8)])
@pytest.mark.parametrize("group_top", [1, 2, 3])
def test_route_groups_of_special_values(E, groups, group_top):
    """A group's value is a sum of its largest: NaN where one of them is or where infinities of both signs meet,
    and NaN counts as the largest, before infinity; ties to the lowest group."""
    per, inf, nan = E // groups, float("inf"), float("nan")
    x, bias = torch.zeros(3, E), torch.zeros(3, E)
    x[0, 2 * per + 3] = nan                              # a NaN, and an infinity in an earlier group
    bias[0, 1] = inf
    bias[1, :per] = inf                                  # infinities, the later of two groups the better otherwise
    bias[1, per:2 * per] = inf
    bias[1, 2 * per:] = 100.0
    bias[2, 2 * per:3 * per] = -inf                      # both signs: NaN where two values or more count
    bias[2, 2 * per + 4] = inf
    bias[2, 1] = inf
    first = [2 * per + 3, 0, 1 if group_top == 1 else 2 * per + 4]
    r = dg.router(2, "sigmoid", groups=groups, top_groups=1, group_top=group_top)
    for i in range(3):
        index, _ = dg.gemm_experts_route_tensors(x[i:i + 1].cuda(), r, bias[i].cuda())
        got = index[0].tolist()
        assert got[0] == first[i] and got[0] // per == got[1] // per, (i, got)
