"""Routing by groups: groups' scores that cancel, groups of whole warps with masked
experts, groups in which nobody is left."""
import pytest
import torch

import quantized_gemm_tcgen05_gb300 as qg
from test_moe_route_gpu import check, h, normal, ws  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def test_a_sum_that_cancels(h, ws):  # noqa: F811
    """Scores of the second group are larger by 2.9e-5 - 4e-5 + 2.9e-5; at 1000 fp32
    numbers are 6e-5 apart."""
    s = torch.tensor([[0.50004, 0.5, 0.500029, 0.500029]], dtype=torch.float64)
    l = torch.log(s / (1 - s)).float().cuda()
    bias = torch.tensor([1000.0, -1000.0, 1000.0, -1000.0], device="cuda")
    ids, *_ = check(h, ws, l, 1, score="sigmoid", bias=bias, groups=2, group_topk=1, group_best=2)
    assert ids.tolist() == [[2]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [100.0, 1000.0, 30000.0])
@pytest.mark.parametrize("experts,groups,keep", [(16, 8, 3), (24, 6, 2), (256, 8, 4), (128, 2, 1)])
def test_biases_of_both_signs(h, ws, experts, groups, keep, size, score):  # noqa: F811
    """One expert of a group has a large bias, all others its negative: a group's score is
    the small difference of two large numbers."""
    bias = torch.full((experts,), -size)
    bias[::experts // groups] = size
    check(h, ws, normal(experts, 300, experts), 2, score=score, bias=bias.cuda(), groups=groups, group_topk=keep, group_best=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("large", [3.4028234e38, float("inf")])
def test_biases_at_the_ends_of_the_range(h, ws, large, score):  # noqa: F811
    bias = torch.zeros(16)
    bias[3], bias[4], bias[5], bias[9], bias[10], bias[12] = large, -3.4028234e38, -3.4028234e38, large, large, -3.4028234e38
    l = normal(3, 60, 16)
    check(h, ws, l, 5, score=score, bias=bias.cuda())
    check(h, ws, l, 5, score=score, bias=bias.cuda(), groups=8, group_topk=4, group_best=2)
    check(h, ws, l, 5, score=score, bias=bias.cuda(), groups=4, group_topk=2, group_best=1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("experts,groups,keep", [(256, 8, 4), (96, 3, 2), (128, 2, 1), (1024, 16, 5), (512, 4, 4), (160, 5, 3)])
def test_masks_in_groups_of_whole_warps(h, ws, experts, groups, keep, best, biased, score):  # noqa: F811
    """Masked experts, groups with one live expert or none, tokens with fewer live groups
    than are kept."""
    tokens, size = 60, experts // groups
    g = torch.Generator().manual_seed(experts)
    l = normal(experts, tokens, experts).cpu()
    l[torch.rand(tokens, experts, generator=g) < 0.8] = -torch.inf
    by_group = l.view(tokens, groups, size)
    by_group[torch.rand(tokens, groups, generator=g) < 0.4] = -torch.inf  # nobody
    one = torch.rand(tokens, groups, generator=g) < 0.3
    only = torch.where(torch.arange(size) == size // 2, 1.0, -torch.inf)
    by_group[one] = only
    l[0] = -torch.inf
    l[1] = -torch.inf
    l[1, experts - 1] = 0.5  # one live expert at all
    bias = (0.1 * torch.randn(experts, generator=g)) if biased else None
    if biased:
        bias[:size - 1] = -torch.inf  # the first group has its last expert at most
        bias = bias.cuda()
    check(h, ws, l.cuda(), min(8, experts), score=score, bias=bias, groups=groups, group_topk=keep, group_best=best)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,keep", [(256, 8, 4), (128, 2, 1), (1024, 16, 5)])
def test_equal_groups_of_whole_warps(h, ws, experts, groups, keep, score):  # noqa: F811
    """Groups with equal scores: the first ones are kept; a better one behind them."""
    l = torch.zeros(12, experts)
    for t in range(6):
        l[t, experts - 1 - 7 * t] = 0.25
    for best in (1, 2):
        check(h, ws, l.cuda(), 6, score=score, groups=groups, group_topk=keep, group_best=best)
        check(h, ws, l.cuda(), 6, score=score, bias=torch.zeros(experts, device="cuda"), groups=groups, group_topk=keep, group_best=best)
