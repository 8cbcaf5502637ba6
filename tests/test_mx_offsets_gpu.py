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
