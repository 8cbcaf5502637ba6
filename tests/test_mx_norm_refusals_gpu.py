"""What gemm_mx_norm_quantize refuses of a gate's row stride: the range is that of
every other stride, checked before a kernel sees it."""
import pytest
import torch

import quantized_gemm_tcgen05_gb300 as qg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ld", [(1 << 40) + 1, 1 << 62, -(1 << 40), 2 ** 63 - 1])
def test_gate_stride_out_of_range(ld):
    h = qg.gemm_create()
    r = torch.ones(1, 128, dtype=torch.float16, device="cuda")  # one row: the stride is not used
    out, o = torch.full_like(r, 4.0), qg.MxOperand(qg.GEMM_NVFP4, 1, 128)
    n = qg.gemm_mx_norm_t(format=qg.GEMM_NVFP4, tensor_scale=1.0, eps=1e-5, residual_scale=1.0, gate=qg.ptr(r),
                          gate_type=qg.GEMM_F16, gate_ld=ld)
    rc = qg.gemm_mx_norm_quantize(h, n, qg.ptr(r), qg.row_major(r), qg.ptr(r), qg.row_major(r), qg.ptr(out), qg.row_major(out),
                                  *o.args(), qg.current_stream())
    torch.cuda.synchronize()
    assert rc == qg.GEMM_ERR_INVALID_ARG and bool((out == 4).all())
    qg.gemm_destroy(h)
