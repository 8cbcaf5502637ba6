"""GPU tests of 4-bit products without K: D = act(beta C + bias), for a grouped
product of the rows that an expert holds, and of no others."""
import pytest
import torch

import quantized_gemm_tcgen05_gb300 as qg

pytestmark = pytest.mark.gpu

ACTS = {"": 0, "bias": 1, "relu": 1 | qg.GEMM_EPILOGUE_RELU, "gelu": 1 | qg.GEMM_EPILOGUE_GELU}


@pytest.fixture(scope="module")
def h():
    h = qg.gemm_create()
    yield h
    qg.gemm_destroy(h)


def without_k(h, c, beta, act, bias, off=None, out=None):
    m, n = c.shape
    e = torch.zeros(64, dtype=torch.uint8, device="cuda")
    op = qg.gemm_op_t(epilogue=ACTS[act], bias=qg.ptr(bias) if act else None, bias_type=qg.GEMM_F32)
    out = torch.full((m, n), 9.0, dtype=c.dtype, device="cuda") if out is None else out
    E = 0 if off is None else off.numel() - 1
    a, b = qg.layout(qg.GEMM_E2M1, 0, m, 0, 32), qg.layout(qg.GEMM_E2M1, 1, 0, n, 32, max(E, 1), 32 * n)
    args = (qg.ptr(e), a, qg.ptr(e), 0, qg.ptr(e), b, qg.ptr(e), 0, beta, qg.ptr(c), qg.row_major(c), qg.ptr(out),
            qg.row_major(out))
    if E:
        rc = qg.gemm_run_mx_grouped(h, op, qg.GEMM_NVFP4, float("inf"), None, *args, qg.ptr(off), E, qg.current_stream())
    else:
        rc = qg.gemm_run_mx(h, op, qg.GEMM_NVFP4, float("inf"), *args, qg.current_stream())
    assert rc == 0, qg.gemm_status_string(rc)
    assert qg.gemm_last_choice(h) == "scale_c"
    return out


def expected(c, beta, act, bias):
    x = beta * c.double() + (bias.double() if act else 0.0)
    return torch.relu(x) if act == "relu" else x * 0.5 * torch.special.erfc(-x / 2 ** 0.5) if act == "gelu" else x


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("beta", [0.0, 0.75])
@pytest.mark.parametrize("off", [None, [0, 5, 5, 40], [3, 10, 10, 31], [0, 0, 0, 0]])
def test_rows_written(h, dtype, act, beta, off):
    m, n = 40, 301
    g = torch.Generator().manual_seed(1)
    c, bias = (2 * torch.randn(m, n, generator=g)).to(dtype).cuda(), (2 * torch.randn(n, generator=g)).cuda()
    lo, hi = (0, m) if off is None else (off[0], off[-1])
    offd = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    out = without_k(h, c, beta, act, bias, offd)
    want = expected(c, beta, act, bias)[lo:hi]
    # fp32: beta c, the sum and the activation's rounding (of |x| <= 16: 1e-5 covers
    # all of it, 16 * 8 * 2^-24), then half a unit of the type
    unit = {torch.float32: 0.0, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[dtype]
    assert bool(((out[lo:hi].double() - want).abs() <= 1e-5 + unit * want.abs()).all())
    assert bool((out[:lo] == 9).all()) and bool((out[hi:] == 9).all())
    # in place
    same = without_k(h, c, beta, act, bias, offd, out=c) if beta else out
    assert torch.equal(same[lo:hi], out[lo:hi])
