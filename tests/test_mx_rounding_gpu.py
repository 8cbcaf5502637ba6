"""GPU tests of tensor scales that are no powers of two: quantisation, where s g
and the quotients are rounded, and its inverse, whose values are rounded once.
All comparisons are exact."""
import numpy as np
import pytest
import torch

import mx_ref as R
import quantized_gemm_tcgen05_gb300 as qg

pytestmark = pytest.mark.gpu

NV = qg.GEMM_NVFP4
BITS = {torch.float16: 11, torch.bfloat16: 8, torch.float32: 24}


@pytest.fixture(scope="module")
def h():
    h = qg.gemm_create()
    yield h
    qg.gemm_destroy(h)


def rounded(x, bits):
    """To `bits` significant bits, ties to even (x exact in 64 bits, no
    subnormal result)."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(np.ldexp(m, bits)), e - bits)


def every_value():
    """One row per positive scale byte, all sixteen codes: a block each."""
    byte = np.arange(1, 127, dtype=np.uint8)[:, None]
    return np.tile(np.arange(16, dtype=np.uint8), (126, 1)), byte


def awkward_scales(bits):
    """fp32 tensor scales for which some code * scale * g lies so near a tie of
    `bits` bits that its fp32 rounding lies on it."""
    code, byte = every_value()
    exact = np.unique(np.abs(R.VALUES[code] * R.scale_values(byte, R.NVFP4)))[1:]
    frac = np.unique(np.frexp(exact)[0])  # the significands there are
    out = []
    for f in frac:
        for tie in range(2 ** (bits - 1), 2 ** bits):
            # (tie + 1/2 + a little) / f, as fp32
            g = np.float32((tie + 0.5 + 2.0 ** (bits - 26)) / 2.0 ** bits / f)
            p = f * np.float64(g)
            if rounded(rounded(p, 24), bits) != rounded(p, bits):
                out.append(float(g))
    return out


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_inverse_is_rounded_once(h, dtype):
    scales = awkward_scales(BITS[dtype])
    assert len(scales) >= 20
    code, byte = every_value()
    rows, k = code.shape
    o = qg.MxOperand(NV, rows, k)
    o.codes.copy_(torch.from_numpy(R.pack(code)))
    o.scales[:R.tile(byte).size].copy_(torch.from_numpy(R.tile(byte)))
    for pad in (0, 3):  # rows on 16-byte boundaries, and not
        for g in scales[::max(1, len(scales) // 40)]:
            out = torch.empty(rows, k + pad, dtype=dtype, device="cuda")[:, :k]
            assert qg.gemm_mx_dequantize(h, NV, g, *o.args(), qg.ptr(out), qg.row_major(out), None, 0,
                                         qg.current_stream()) == 0
            want = rounded(R.dequantize(code, byte, NV, np.float64(np.float32(g))), BITS[dtype])
            normal = np.abs(want) >= float(torch.finfo(dtype).smallest_normal)  # (and what no code is: zero)
            got = out.double().cpu().numpy()
            assert np.array_equal(got[normal], want[normal]), g


def expected(x, g):
    """gemm_mx_quantize's NVFP4 with every step rounded to fp32, in fp32."""
    f = np.float32
    rows, k = x.shape
    nb = R.ceil(k, 16)
    v = np.zeros((rows, nb * 16), f)
    v[:, :k] = x
    v = v.reshape(rows, nb, 16)
    t = np.minimum(np.abs(v).max(-1) / (f(6) * f(g)), f(448))
    byte = R.nearest(R.e4m3_values()[:127], t)
    u = (R.e4m3_values()[byte].astype(f) * f(g)).astype(f)
    w = np.where(u[..., None] > 0, v / np.where(u > 0, u, f(1))[..., None], f(0))
    assert w.dtype == f and t.dtype == f
    code = R.nearest(R.MAG, np.abs(w)) + 8 * np.signbit(w)
    return code.reshape(rows, -1)[:, :k].astype(np.uint8), byte.astype(np.uint8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("g", [0.001, 1 / 3, 0.7, 3.3e-5, 5.0, 12345.678, 1.9999998807907104, 2.0 ** -64, 2.0 ** 64])
def test_quantise(h, dtype, g):
    rows, k = 300, 1040
    gen = torch.Generator().manual_seed(5)
    x = torch.randn(rows, k, generator=gen) * torch.exp(3 * torch.randn(rows, 1, generator=gen))
    if dtype != torch.float16:
        x = x * g  # the range such a tensor scale is made for
    if dtype == torch.float32:
        # and, in the lower rows, values that sit on the ties of their block's grid
        u = (torch.from_numpy(R.e4m3_values()[:127]).float()[torch.randint(8, 127, (100, k // 16), generator=gen)]
             * np.float32(g)).repeat_interleave(16, 1)
        tie = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])[torch.randint(0, 8, (100, k), generator=gen)]
        tie[:, ::16] = 6.0
        x[200:] = tie * u
    x = x.to(dtype).cuda()
    o = qg.MxOperand(NV, rows, k)
    assert qg.gemm_mx_quantize(h, NV, g, qg.ptr(x), qg.row_major(x), *o.args(), None, 0, qg.current_stream()) == 0
    code, byte = expected(x.float().cpu().numpy(), g)
    assert np.array_equal(o.scales.cpu().numpy()[:R.tile(byte).size].reshape(-1)[R.scale_at(
        np.arange(rows)[:, None], np.arange(byte.shape[1])[None], R.ceil(byte.shape[1], 4))], byte)
    assert np.array_equal(R.unpack(o.codes.cpu().numpy(), k), code)
