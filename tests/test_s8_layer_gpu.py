"""The int8 mixture-of-experts example step by step, each from what the step before it
wrote, and its result as a whole against the layer in 64 bits: as far off as int8 makes
it, which is a small part of what the experts add."""
import os
import sys

import numpy as np
import pytest
import torch

import moe_ref as ref
import quantized_gemm_tcgen05_gb300 as qg

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import s8_moe  # noqa: E402

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def gelu(x):
    return 0.5 * x * torch.special.erfc(-x / 2 ** 0.5)


def run(tokens, hidden, inner, experts, topk):
    h = qg.gemm_create()
    w = s8_moe.Weights(h, hidden, inner, experts)
    layer = s8_moe.Layer(h, w, tokens, topk)
    x = torch.randn(tokens, hidden, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    layer.step(x)
    assert qg.gemm_device_status(h, qg.current_stream()) == qg.GEMM_OK
    qg.gemm_destroy(h)
    return w, layer, x


@pytest.mark.parametrize("tokens,hidden,inner,experts,topk", [(1, 256, 384, 8, 2), (37, 272, 400, 8, 2), (300, 512, 768, 16, 4)])
def test_steps(tokens, hidden, inner, experts, topk):
    w, layer, x = run(tokens, hidden, inner, experts, topk)
    # the router's logits: the library's rule for its products
    full, size = (f(x.double()) @ f(w.router.double()).t() for f in (lambda t: t, torch.abs))
    assert ((layer.logits.double() - full).abs() <= 1e-5 * size + 1e-6 + full.abs() * 2.0 ** -8 * 1.01).all()
    ids, weights, rows, offsets = ref.route(layer.logits.double().cpu().numpy(), topk, score="sigmoid", bias=w.router_bias.cpu().numpy())
    for got, want in ((layer.ids, ids), (layer.rows, rows), (layer.offsets, offsets)):
        assert np.array_equal(got.cpu().numpy(), want)
    # exponentials of 2 units, a sum of topk, a quotient, a product
    assert (np.abs(layer.weights.double().cpu().numpy() - weights) <= (topk + 8) * 2.0 ** -23 * weights).all()
    q, s = ref.quantize(x)
    for t in range(tokens):
        for r in rows[t]:
            assert np.array_equal(layer.x8[r].cpu().numpy(), q[t]) and float(layer.x_scale[r]) == float(s[t])
    for e in range(experts):
        mine = slice(int(offsets[e]), int(offsets[e + 1]))
        if offsets[e] == offsets[e + 1]:
            continue
        pre = ref.product(ref.sums(layer.x8[mine], w.up[e]), 1.0, layer.x_scale[mine], w.up_scale[e], torch.float32, bias=w.up_bias).double()
        y, got = gelu(pre), layer.mid[mine].double().cpu()
        assert ((got - y).abs() <= y.abs() * (2e-5 + 2.0 ** -8 * 1.0001) + 2.0 ** -25).all()
        down = ref.product(ref.sums(layer.mid8[mine], w.down[e]), 1.0, layer.mid_scale[mine], w.down_scale[e], BF16)
        assert torch.equal(layer.out_rows[mine].cpu(), down)
    q, s = ref.quantize(layer.mid)
    assert np.array_equal(layer.mid8.cpu().numpy(), q) and np.array_equal(layer.mid_scale.cpu().numpy(), s)
    terms = layer.weights.double().unsqueeze(-1) * layer.out_rows.double()[layer.rows.long()]
    total, size = terms.sum(1) + x.double(), terms.abs().sum(1) + x.double().abs()
    # topk + 1 fused steps, one rounding
    assert ((layer.out.double() - total).abs() <= (topk + 1) * 2.0 ** -24 * size * 1.01 + total.abs() * 2.0 ** -8 * 1.01).all()


@pytest.mark.parametrize("tokens,hidden,inner,experts,topk", [(64, 256, 384, 8, 2), (300, 512, 768, 16, 4)])
def test_whole(tokens, hidden, inner, experts, topk):
    w, layer, x = run(tokens, hidden, inner, experts, topk)
    ids, weight = layer.ids.long(), layer.weights.double()
    up, down = (q.double() * s.double().unsqueeze(-1) for q, s in ((w.up, w.up_scale), (w.down, w.down_scale)))
    want, var = x.double(), torch.zeros_like(x, dtype=torch.float64)
    for j in range(topk):
        r = layer.rows[:, j].long()
        pre = torch.einsum("th,tih->ti", x.double(), up[ids[:, j]]) + w.up_bias.double()
        mid = gelu(pre)
        want = want + weight[:, j:j + 1] * torch.einsum("ti,thi->th", mid, down[ids[:, j]])
        # A code is off by up to half a scale, evenly: scale^2 / 12 on average, each by
        # itself; GELU's slope is below 1.13; bf16 rounds by 2^-9 on average at most.
        ex = (layer.x_scale[r].double() ** 2 / 12).unsqueeze(1) * (up[ids[:, j]] ** 2).sum(2)
        em = 1.13 ** 2 * ex + (mid * 2.0 ** -9) ** 2 + (layer.mid_scale[r].double() ** 2 / 12).unsqueeze(1)
        y = torch.einsum("ti,thi->th", em, down[ids[:, j]] ** 2)
        var = var + weight[:, j:j + 1] ** 2 * (y + (layer.out_rows[r].double() * 2.0 ** -9) ** 2)
    var = var + (want * 2.0 ** -9) ** 2
    # tens of thousands of errors: their mean square is near the expected one; rows of one
    # expert share no errors, tokens' topk rows share those of x (at most topk times the variance)
    off, limit = (layer.out.double() - want).square().mean().sqrt(), (topk * var.mean()).sqrt() * 1.1
    added = (want - x.double()).square().mean().sqrt()
    assert off <= limit and limit < 0.1 * added, (off, limit, added)
