"""The int8 mixture-of-experts example: its step against the layer in 64 bits, and
the script as it is run."""
import os
import subprocess
import sys

import pytest
import torch

import quantized_gemm_tcgen05_gb300 as qg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
import s8_moe  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,hidden,inner,experts,topk", [(1, 256, 384, 8, 2), (37, 272, 400, 8, 2), (500, 512, 768, 16, 4)])
def test_layer(tokens, hidden, inner, experts, topk):
    h = qg.gemm_create()
    w = s8_moe.Weights(h, hidden, inner, experts)
    layer = s8_moe.Layer(h, w, tokens, topk)
    x = torch.randn(tokens, hidden, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    out = layer.step(x).double()
    assert qg.gemm_device_status(h, qg.current_stream()) == qg.GEMM_OK
    # in 64 bits, from the layer's logits and quantised weights
    s = torch.sigmoid(layer.logits.double())
    ids = torch.argsort(-(s + w.router_bias.double()), dim=1, stable=True)[:, :topk]
    assert torch.equal(ids.int(), layer.ids)
    weight = s.gather(1, ids)
    weight = weight / weight.sum(1, keepdim=True)
    up = w.up.double() * w.up_scale.double().unsqueeze(-1)
    down = w.down.double() * w.down_scale.double().unsqueeze(-1)
    want, size = x.double(), x.double().abs()
    xd = x.double()
    for j in range(topk):
        pre = torch.einsum("th,tih->ti", xd, up[ids[:, j]]) + w.up_bias.double()
        mid = pre * torch.special.ndtr(pre)
        y = torch.einsum("ti,thi->th", mid, down[ids[:, j]])
        want = want + weight[:, j:j + 1] * y
        # An int8 code is off by at most half a scale: amax / 254 of its row.  A row of x of
        # norm |x| and hidden elements is off by at most amax(x) / 254 sqrt(hidden) in norm, and
        # so is each entry of its product by that times the norm of the matrix' row; GELU's
        # slope is below 1.13.  The middle rows likewise, and bf16 roundings of 2^-8.
        ex = xd.abs().amax(1, keepdim=True) / 254 * hidden ** 0.5 * up[ids[:, j]].norm(dim=2)
        em = 1.13 * ex + mid.abs() * 2.0 ** -8
        top = (mid.abs() + em).amax(1, keepdim=True)
        row = em.norm(dim=1, keepdim=True) + top / 254 * inner ** 0.5
        err = row * down[ids[:, j]].norm(dim=2)
        size = size + weight[:, j:j + 1] * (err * 2 ** 8 + y.abs() + err)
    assert ((out - want).abs() <= size * 2.0 ** -8 * 1.01).all()
    qg.gemm_destroy(h)


def test_script_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "s8_moe.py"), "--tokens", "100", "--hidden", "256", "--inner", "512"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "us a layer" in r.stdout, r.stdout + r.stderr


def test_block_example_routes():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "mx_block.py"), "--tokens", "40", "--hidden", "256", "--inner", "512",
                        "--experts", "8"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "us a block" in r.stdout, r.stdout + r.stderr
