"""GPU tests of expert offsets that are no partition of the rows: the calls come
back soon, nothing outside D, the codes and the scales is read or written."""
import numpy as np
import pytest
import torch

import mx_ref as R
import quantized_gemm_tcgen05_gb300 as qg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h():
    h = qg.gemm_create()
    yield h
    qg.gemm_destroy(h)


def dev32(off):
    return torch.from_numpy(np.asarray(off, dtype=np.int64).astype(np.int32)).cuda()


# one expert that promises 2^31 rows, negative and falling offsets, all of them at once
WILD = [[0, 2 ** 31 - 1, 5, 300], [-2 ** 31, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1], [300, 200, 100, 0], [-5, 40, 2 ** 30, 300]]


@pytest.mark.parametrize("pin", ["mx_bn64", "mx_bn128", "mx2_bn256"])
@pytest.mark.parametrize("off", WILD, ids=range(len(WILD)))
def test_product_comes_back_and_stays_inside(h, monkeypatch, pin, off):
    monkeypatch.setenv("GEMM_FORCE_KERNEL", pin)
    fmt, rows, n, k, E = qg.GEMM_NVFP4, 300, 512, 4096, 3
    a, w = qg.MxOperand(fmt, rows, k, num_experts=E), qg.MxOperand(fmt, n, k, num=E)
    offd = dev32(off)
    buf = torch.full((rows + 600, n), 5.0, dtype=torch.bfloat16, device="cuda")
    out = buf[300:300 + rows]

    def call():
        rc = qg.gemm_run_mx_grouped(h, qg.gemm_op_t(), fmt, 1.0, None, *a.args(), *w.args(b=True), 0.0, None, None,
                                    qg.ptr(out), qg.row_major(out), qg.ptr(offd), E, qg.current_stream())
        assert rc == 0

    call()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    call()
    end.record()
    assert qg.gemm_device_status(h, qg.current_stream()) == 0
    assert bool((buf[:300] == 5).all()) and bool((buf[300 + rows:] == 5).all())
    # six row blocks at most, some tens of microseconds; 2^31 rows would take a second
    assert start.elapsed_time(end) < 20.0


@pytest.mark.parametrize("fmt", [qg.GEMM_NVFP4, qg.GEMM_MXFP4])
def test_rows_without_scales_are_left_out(h, fmt):
    # offsets whose experts before the last claim four of the five atom rows that
    # 256 rows by three experts have: rows 8 .. 135 of the last expert find scales,
    # rows 136 .. 255 do not and are neither quantised nor dequantised
    rows, k, E, lo, hi = 256, 96, 3, 8, 136
    offd = dev32([1000, 1512, lo, rows])
    x = torch.randn(rows, k, generator=torch.Generator().manual_seed(3)).cuda()
    o = qg.MxOperand(fmt, rows, k)
    size = qg.gemm_mx_scale_size(fmt, rows, k, E)
    scales = torch.full((size + 4096,), 0xAA, dtype=torch.uint8, device="cuda")
    o.codes.fill_(0xAA)
    c, cl, _, _ = o.args()
    assert qg.gemm_mx_quantize(h, fmt, 1.0, qg.ptr(x), qg.row_major(x), c, cl, qg.ptr(scales), size, qg.ptr(offd), E,
                               qg.current_stream()) == 0
    code, byte = R.quantize(x.double().cpu().numpy(), fmt)
    got = o.codes.cpu().numpy()
    assert np.array_equal(got[lo:hi], R.pack(code[lo:hi])) and (got[:lo] == 0xAA).all() and (got[hi:] == 0xAA).all()
    want = R.tile(byte[lo:hi], 4 * 128 + np.arange(hi - lo), size // (512 * R.ceil(k, 4 * R.BLOCK[fmt])), fill=0xAA)
    assert np.array_equal(scales.cpu().numpy()[:size], want) and bool((scales[size:] == 0xAA).all())
    o.codes.copy_(torch.from_numpy(R.pack(code)))
    out = torch.full((rows, k), 7.0, device="cuda")
    assert qg.gemm_mx_dequantize(h, fmt, 1.0, c, cl, qg.ptr(scales), size, qg.ptr(out), qg.row_major(out), qg.ptr(offd), E,
                                 qg.current_stream()) == 0
    assert np.array_equal(out[lo:hi].double().cpu().numpy(), R.dequantize(code, byte, fmt)[lo:hi])
    assert bool((out[:lo] == 7).all()) and bool((out[hi:] == 7).all())


@pytest.mark.parametrize("off", WILD, ids=range(len(WILD)))
def test_quantisation_and_norm_stay_inside(h, off):
    fmt, rows, k, E = qg.GEMM_NVFP4, 300, 200, 3
    offd = dev32(off)
    size = qg.gemm_mx_scale_size(fmt, rows, k, E)
    x = torch.randn(rows, k, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    scales = torch.full((size + 8192,), 0xAA, dtype=torch.uint8, device="cuda")
    at, o = 4096, qg.MxOperand(fmt, rows, k)
    c, cl, _, _ = o.args()
    assert qg.gemm_mx_quantize(h, fmt, 1.0, qg.ptr(x), qg.row_major(x), c, cl, qg.ptr(scales) + at, size, qg.ptr(offd), E,
                               qg.current_stream()) == 0
    n = qg.gemm_mx_norm_t(format=fmt, tensor_scale=1.0, eps=1e-5, residual_scale=1.0, expert_offsets=qg.ptr(offd),
                          num_experts=E)
    assert qg.gemm_mx_norm_quantize(h, n, None, None, qg.ptr(x), qg.row_major(x), None, None, c, cl, qg.ptr(scales) + at, size,
                                    qg.current_stream()) == 0
    out = torch.full((rows + 20, k), 7.0, device="cuda")
    y = out[10:10 + rows]
    assert qg.gemm_mx_dequantize(h, fmt, 1.0, c, cl, qg.ptr(scales) + at, size, qg.ptr(y), qg.row_major(y), qg.ptr(offd), E,
                                 qg.current_stream()) == 0
    assert bool((scales[:at] == 0xAA).all()) and bool((scales[at + size:] == 0xAA).all())
    assert bool((out[:10] == 7).all()) and bool((out[-10:] == 7).all())
