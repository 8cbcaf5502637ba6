"""GPU tests of the values the 4-bit products' epilogues store: GELU over its
whole range, and that a value depends neither on the kernel, nor on its place
in D, nor on D's alignment.

Tolerance of GELU.  For a 16-bit D the value before the rounding is within
2e-5 of x Phi(x), relative (the fitted tail 3e-7, the exponential of an
argument of up to 85 with three roundings to fp32, 85 * 2.5 * 2^-24 = 1.3e-5, and
the approximate exponential and reciprocal 2^-21 each), or below fp32's normal numbers; the rounding
adds half a unit of D.  For an fp32 D 1 + erf is right to three units of fp32
at 2 (3 * 2^-23, erff's bound of two and the sum's rounding), which times
0.5 |x| with two more roundings of x's argument and of the products stays
below 4 * 2^-23 |x|."""
import numpy as np
import pytest
import torch

import mx_ref as R
import oracle
import quantized_gemm_tcgen05_gb300 as qg
import synth

pytestmark = pytest.mark.gpu

TD = {synth.F32: torch.float32, synth.F16: torch.float16, synth.BF16: torch.bfloat16}
KERNELS = ["mx_bn64", "mx_bn128", "mx2_bn256"]
GELU = qg.GEMM_EPILOGUE_BIAS | qg.GEMM_EPILOGUE_GELU


@pytest.fixture(scope="module")
def h():
    h = qg.gemm_create()
    yield h
    qg.gemm_destroy(h)


def operand(fmt, rows, k, code, byte):
    o = qg.MxOperand(fmt, rows, k)
    o.codes.copy_(torch.from_numpy(R.pack(code)))
    flat = R.tile(byte)
    o.scales[:flat.size].copy_(torch.from_numpy(flat))
    return o


def product(h, fmt, a, b, d, ldd=None, off=0, c=None, beta=0.0, alpha=1.0, **op):
    """D as a view into a buffer, `off` elements in, row stride ldd."""
    m, n = a.rows, b.rows
    ldd = n if ldd is None else ldd
    buf = torch.full((m * ldd + off,), 9.0, dtype=TD[d], device="cuda")
    out = buf[off:].view(m, ldd)[:, :n]
    rc = qg.gemm_run_mx(h, qg.gemm_op_t(**op), fmt, alpha, *a.args(), *b.args(b=True), beta, qg.ptr(c),
                        None if c is None else qg.row_major(c), qg.ptr(out), qg.layout(d, 0, m, n, ldd),
                        qg.current_stream())
    assert rc == 0, qg.gemm_status_string(rc)
    assert qg.gemm_device_status(h, qg.current_stream()) == 0
    return out


def arguments(n):
    """GELU's argument for each of n columns: near zero, the middle, the tails."""
    far = [-30.0, -1000.0, -30000.0, -1e6, -1e30, 30.0, 1000.0, 30000.0, 1e6, 1e30, 0.0, -0.0]
    near = [s * 2.0 ** -e for e in range(1, 30, 4) for s in (1, -1)]
    rest = n - len(far) - len(near)
    x = np.concatenate([far, near, np.linspace(-14, 14, rest)])
    return torch.from_numpy(np.random.default_rng(n).permutation(x)).float().cuda()


@pytest.mark.parametrize("d", [synth.BF16, synth.F16, synth.F32])
@pytest.mark.parametrize("form", ["aligned", "with C", "odd stride", "odd start", "k slices"])
@pytest.mark.parametrize("pin", KERNELS)
def test_gelu_over_its_range(h, monkeypatch, pin, form, d):
    # codes are zero, so the bias alone is GELU's argument
    if form == "k slices" and pin == "mx2_bn256":
        pytest.skip("the CTA-pair kernel does not slice K")
    monkeypatch.setenv("GEMM_FORCE_KERNEL", pin)
    fmt, m, n, k = qg.GEMM_NVFP4, 130, 768, 512
    a, b = qg.MxOperand(fmt, m, k), qg.MxOperand(fmt, n, k)
    x = arguments(n)
    kw = dict(epilogue=GELU, bias=qg.ptr(x), bias_type=qg.GEMM_F32)
    if form == "with C":
        kw.update(c=torch.zeros(m, n, dtype=TD[d], device="cuda"), beta=1.0)
    if form == "odd stride":
        kw.update(ldd=n + 1)
    if form == "odd start":
        kw.update(off=1)
    if form == "k slices":
        kw.update(splitk=2)
    out = product(h, fmt, a, b, d, **kw)
    assert torch.equal(out, out[:1].expand_as(out))
    got, v = out[0].double().cpu().numpy(), x.double().cpu().numpy()
    want = (x.double() * 0.5 * torch.special.erfc(-x.double() / 2 ** 0.5)).cpu().numpy()
    if d == synth.F32:
        tol = 4 * 2.0 ** -23 * np.abs(v)
    else:
        top = float(torch.finfo(TD[d]).max)
        fits = np.abs(want) <= top  # f16: beyond, infinity
        assert (got[~fits] == np.inf).all()
        got, want = got[fits], want[fits]
        tol = 2e-5 * np.abs(want) + 2.0 ** -126 + 0.5 * oracle.ulp(d, want)
    assert (np.abs(got - want) <= tol).all(), list(zip(v[:9], got[:9], want[:9]))


@pytest.mark.parametrize("d", [synth.BF16, synth.F16, synth.F32])
def test_gelu_of_infinities_and_nan(h, d):
    # as 0.5 x (1 + erf): inf, NaN for -inf (-inf * 0) and NaN
    fmt = qg.GEMM_NVFP4
    a, b = qg.MxOperand(fmt, 3, 64), qg.MxOperand(fmt, 64, 64)
    x = torch.zeros(64, device="cuda")
    x[5], x[6], x[40] = float("inf"), float("-inf"), float("nan")
    out = product(h, fmt, a, b, d, epilogue=GELU, bias=qg.ptr(x), bias_type=qg.GEMM_F32)
    assert bool((out[:, 5] == float("inf")).all()) and bool(out[:, 6].isnan().all()) and bool(out[:, 40].isnan().all())
    assert int((out == 0).sum()) == 3 * 61


@pytest.mark.parametrize("d", [synth.BF16, synth.F16])
@pytest.mark.parametrize("epilogue", [0, 1, 1 | qg.GEMM_EPILOGUE_RELU, GELU])
@pytest.mark.parametrize("beta", [0.0, 0.75])
def test_value_does_not_depend_on_its_place(h, monkeypatch, d, epilogue, beta):
    # sums of few products with scales of 1 are exact in any order, so D has the
    # same bits from every kernel, K slicing and form of the epilogue
    fmt, m, n, k = qg.GEMM_MXFP4, 150, 512, 512
    rng = np.random.default_rng(7)
    a, b = (operand(fmt, r, k, rng.integers(0, 16, (r, k)).astype(np.uint8), np.full((r, k // 32), 127, np.uint8))
            for r in (m, n))
    bias = torch.randn(n, generator=torch.Generator().manual_seed(1)).cuda()
    c = torch.randn(m, n, generator=torch.Generator().manual_seed(2)).to(TD[d]).cuda() if beta else None
    op = dict(epilogue=epilogue, bias=qg.ptr(bias) if epilogue else None, bias_type=qg.GEMM_F32, c=c, beta=beta,
              alpha=0.013)
    want = None
    for pin in KERNELS:
        monkeypatch.setenv("GEMM_FORCE_KERNEL", pin)
        for kw in [{}, dict(ldd=n + 1), dict(off=1), dict(ldd=n + 16)] + ([dict(splitk=2)] if pin == "mx_bn64" else []):
            got = product(h, fmt, a, b, d, **op, **kw)
            want = got.clone() if want is None else want
            assert torch.equal(got, want), (pin, kw)
