"""Routing where the experts' order hangs on what fp32 cannot hold: runs of equal
candidates at the last slot, next to others that only 64 bits tell apart."""
import pytest
import torch

import quantized_gemm_tcgen05_gb300 as qg
from test_moe_route_gpu import check, h, ws  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def test_equal_candidates_at_the_last_slot(h, ws):  # noqa: F811
    """Two equal candidates share the last slot's score; a third one's is larger, by less
    than fp32 shows."""
    # sigmoid: all three are 1 in fp32
    ids, *_ = check(h, ws, torch.tensor([[18.0, 18.0, 20.0]], device="cuda"), 1, score="sigmoid", bias=torch.zeros(3, device="cuda"))
    assert ids.tolist() == [[2]]
    # softmax: all but the first are 0.1 in fp32
    l = torch.full((1, 40), -1.0, device="cuda")
    l[0, :4] = torch.tensor([24.0, 0.0, 0.0, 1.0])
    ids, *_ = check(h, ws, l, 2, score="softmax", bias=torch.full((40,), 0.1, device="cuda"))
    assert ids.tolist() == [[0, 3]]


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("bias", [0.0, 0.1, -3.0, 1000.0])
@pytest.mark.parametrize("experts,topk", [(3, 1), (8, 2), (24, 6), (33, 8), (60, 4), (256, 8), (300, 32)])
def test_logits_of_a_few_values_and_one_bias(h, ws, experts, topk, bias, x):  # noqa: F811
    """Long runs of equals, saturated (sigmoid) or beside one logit that has nearly all of
    the sum (softmax).  In 64 bits the values' scores lie far apart (e^-22 - e^-24 is
    2e-10, 64-bit numbers at 1000 are 1.2e-13 apart)."""
    g = torch.Generator().manual_seed(experts)
    b = torch.full((experts,), bias, device="cuda")
    kind = {"f32": torch.float32, "bf16": torch.bfloat16}[x]
    # mostly the lowest value, so that the larger ones lie somewhere behind equals
    pick = torch.multinomial(torch.tensor([8.0, 2.0, 1.0, 0.5]), 150 * experts, replacement=True, generator=g).view(150, experts)
    saturated = torch.tensor([18.0, 20.0, 22.0, 24.0])[pick]
    check(h, ws, saturated.to(kind).cuda(), topk, score="sigmoid", bias=b)
    beside = torch.tensor([0.0, 0.5, 1.0, 2.0])[pick]
    beside[:, 0] = 24.0
    check(h, ws, beside.to(kind).cuda(), topk, score="softmax", bias=b)
    if experts % 4 == 0:
        check(h, ws, saturated.to(kind).cuda(), min(topk, experts // 4), score="sigmoid", bias=b, groups=4, group_topk=2, group_best=1)
        check(h, ws, beside.to(kind).cuda(), min(topk, experts // 4), score="softmax", bias=b, groups=4, group_topk=2, group_best=2)


def test_equals_beyond_what_a_warp_holds(h, ws):  # noqa: F811
    """More equal candidates than lanes, a better one behind them."""
    l = torch.full((9, 200), 18.0, device="cuda")
    for t in range(9):
        l[t, 20 * t + 30] = 20.0
    ids, *_ = check(h, ws, l, 3, score="sigmoid", bias=torch.zeros(200, device="cuda"))
    assert ids.tolist() == [[20 * t + 30, 0, 1] for t in range(9)]
