"""Scales of rows that gemm_moe_dispatch copies: an S that nothing would be written
to is refused, and the scales of int8 rows are placed as rows of one column."""
import pytest
import torch

import quantized_gemm_tcgen05_gb300 as qg
from test_moe_rows_gpu import h, place, quantize, values  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def dispatch(h, x, rows, topk, y, s=None):  # noqa: F811
    return qg.gemm_moe_dispatch(h, qg.ptr(x), qg.row_major(x), qg.ptr(rows), topk, qg.ptr(y), qg.row_major(y), qg.ptr(s), qg.current_stream())


@pytest.mark.parametrize("kind", [torch.int8, torch.bfloat16, torch.float32, torch.float8_e4m3fn])
@pytest.mark.parametrize("tokens,rows", [(5, 10), (0, 10), (5, 0)])
def test_scales_that_would_not_be_written(h, kind, tokens, rows):  # noqa: F811
    x, y = torch.zeros(tokens, 64, device="cuda").to(kind), torch.zeros(rows, 64, device="cuda").to(kind)
    m = torch.arange(10, dtype=torch.int32, device="cuda")
    s = torch.full((10,), 9.0, device="cuda")
    assert dispatch(h, x, m, 2, y, s) == qg.GEMM_ERR_INVALID_ARG
    assert dispatch(h, x, m, 2, y) == qg.GEMM_OK
    torch.cuda.synchronize()
    assert (s == 9).all()


@pytest.mark.parametrize("tokens,cols,topk,extra", [(1, 64, 1, 0), (40, 1000, 3, 5), (1030, 33, 8, 0)])
def test_int8_rows_and_their_scales(h, tokens, cols, topk, extra):  # noqa: F811
    """Quantised first and placed then: what placing and quantising in one call gives."""
    x, n = values(tokens, tokens, cols), tokens * topk + extra
    m = place(tokens, tokens, topk, n, 0.1 if extra else 0.0)
    codes, scales = torch.empty(tokens, cols, dtype=torch.int8, device="cuda"), torch.empty(tokens, device="cuda")
    quantize(h, x, codes, scales)
    y, s = torch.full((n, cols), 5, dtype=torch.int8, device="cuda"), torch.full((n, 1), 5.0, device="cuda")
    assert dispatch(h, codes, m, topk, y) == qg.GEMM_OK
    assert dispatch(h, scales.view(-1, 1), m, topk, s) == qg.GEMM_OK
    y2, s2 = torch.full_like(y, 5), torch.full((n,), 5.0, device="cuda")
    assert dispatch(h, x, m, topk, y2, s2) == qg.GEMM_OK
    assert torch.equal(y, y2) and torch.equal(s.view(-1), s2)
