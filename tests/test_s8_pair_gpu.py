"""The CTA-pair int8 product against the one-tile kernel, bit for bit on the device:
many launches over operands that come from far, so that the two CTAs of a pair
finish their halves of the operands at different times."""
import os

import pytest
import torch

import quantized_gemm_tcgen05_gb300 as qg
from test_s8_gemm_gpu import Problem, h, pin  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k,sizes", [(190, 8192, 2048, None), (333, 4096, 1100, None), (64, 20000, 520, None), (700, 2048, 3000, [300, 0, 390, 10])])
def test_halves_of_a_pair(h, pin, m, n, k, sizes):  # noqa: F811
    ps = [Problem(m, n, k, "f32", seed=i, sizes=sizes) for i in range(2)]
    flush = torch.empty(160 << 20, dtype=torch.uint8, device="cuda")
    pin("s8_t128")
    want = [p.run(h).clone() for p in ps]
    assert "t128" in qg.gemm_last_choice(h)
    pin("s8_pair")
    for i in range(30):
        flush.zero_()
        for p, w in zip(ps, want):
            p.out.fill_(7.0)
            p.run(h)
            assert torch.equal(p.out, w), i
    assert "pair" in qg.gemm_last_choice(h)
    os.environ.pop("GEMM_FORCE_KERNEL")
