"""Host-side checks of include/gemm_moe.h and include/gemm_s8.h that need no GPU:
every declared function is exported and bound, and a missing handle is refused."""
import os
import re

import pytest

import quantized_gemm_tcgen05_gb300 as qg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("header,names", [("gemm_moe.h", qg.MOE_SYMBOLS), ("gemm_s8.h", qg.S8_SYMBOLS)])
def test_exports_every_declared_symbol(header, names):
    with open(os.path.join(ROOT, "include", header)) as f:
        declared = set(re.findall(r"^int\s+(gemm_\w+)\s*\(", f.read(), flags=re.M))
    assert declared == set(names)
    for n in names:
        assert hasattr(qg.lib(), n) and hasattr(qg, n)


def test_null_handle_refused():
    op, route = qg.gemm_op_t(), qg.gemm_route_t(topk=1, scale=1.0)
    for rc in (qg.gemm_moe_route(None, route, *[None] * 8), qg.gemm_moe_dispatch(None, None, None, None, 1, None, None, None, None),
               qg.gemm_moe_combine(None, None, None, None, None, 1, 0.0, None, None, None, None, None),
               qg.gemm_s8_quantize(None, *[None] * 6),
               qg.gemm_run_s8(None, op, 1.0, *[None] * 6, 0.0, *[None] * 5),
               qg.gemm_run_s8_grouped(None, op, 1.0, *[None] * 6, 0.0, *[None] * 5, 1, None)):
        assert rc == qg.GEMM_ERR_INVALID_ARG
