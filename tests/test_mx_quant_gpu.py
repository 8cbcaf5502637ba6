"""GPU tests of 4-bit microscaled quantisation and its inverse against numpy in
64 bits: exact codes and scale bytes for every input type, ragged and strided
rows, ties, special values, rows sorted by expert, several matrices."""
import numpy as np
import pytest
import torch

import mx_ref as R
import quantized_gemm_tcgen05_gb300 as qg

pytestmark = pytest.mark.gpu

FORMATS = [qg.GEMM_NVFP4, qg.GEMM_MXFP4]
TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def h():
    h = qg.gemm_create()
    yield h
    qg.gemm_destroy(h)


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)


def quantize(h, x, fmt, g=1.0, counts=None):
    """-> (packed bytes, scale bytes) as numpy, from buffers filled with 0xAA."""
    rows, k = x.shape[-2:]
    num = x.shape[0] if x.dim() == 3 else 1
    E = len(counts) if counts is not None else 0
    o = qg.MxOperand(fmt, rows, k, num_experts=E, num=num)
    o.codes.fill_(0xAA)
    o.scales.fill_(0xAA)
    off = torch.from_numpy(offsets_of(counts).astype(np.int32)).cuda() if E else None
    c, cl, s, sb = o.args()
    rc = qg.gemm_mx_quantize(h, fmt, g, qg.ptr(x), qg.row_major(x), c, cl, s, sb, qg.ptr(off), E, qg.current_stream())
    assert rc == 0, qg.gemm_status_string(rc)
    torch.cuda.synchronize()
    return o, off


def expect(x, fmt, g=1.0, counts=None):
    code, byte = R.quantize(x.double().cpu().numpy(), fmt, g)
    rows, k = code.shape
    packed = R.pack(code)
    packed[:, R.ceil(k, 2):] = 0xAA  # bytes past the row's codes are not written
    if counts is None:
        return packed, R.tile(byte, fill=0xAA)
    return packed, R.tile(byte, R.expert_rows(offsets_of(counts)), rows // 128 + len(counts), fill=0xAA)


def values(rows, k, dtype, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, k, generator=g) * torch.exp(2 * torch.randn(rows, k, generator=g)) * scale
    return x.to(dtype).cuda()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(1, 1), (1, 16), (3, 33), (16, 4096), (129, 64), (200, 1031), (5, 14336), (257, 130), (31, 527)])
def test_exact(h, fmt, dtype, shape):
    x = values(*shape, dtype, seed=shape[0])
    o, _ = quantize(h, x, fmt)
    packed, scales = expect(x, fmt)
    assert np.array_equal(o.scales.cpu().numpy()[:scales.size], scales)
    assert np.array_equal(o.codes.cpu().numpy(), packed)


@pytest.mark.parametrize("g", [0.5, 2.0 ** -10, 4.0])
@pytest.mark.parametrize("dtype", TYPES)
def test_tensor_scale(h, dtype, g):
    x = values(40, 700, dtype, seed=3)
    o, _ = quantize(h, x, qg.GEMM_NVFP4, g)
    packed, scales = expect(x, qg.GEMM_NVFP4, g)
    assert np.array_equal(o.scales.cpu().numpy(), scales)
    assert np.array_equal(o.codes.cpu().numpy(), packed)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("pad,off", [(8, 0), (3, 0), (8, 1), (0, 2)])
def test_strided_and_unaligned_rows(h, fmt, pad, off):
    rows, k = 70, 400
    buf = values(1, rows * (k + pad) + off, torch.bfloat16, seed=9)[0]
    x = buf[off:off + rows * (k + pad)].view(rows, k + pad)[:, :k]
    o, _ = quantize(h, x, fmt)
    packed, scales = expect(x, fmt)
    assert np.array_equal(o.scales.cpu().numpy(), scales) and np.array_equal(o.codes.cpu().numpy(), packed)


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_tie_and_range_end(h, fmt):
    # scale 1 (a 6 in every block), then the grid's midpoints, its points and
    # their fp32 neighbours, both signs
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=np.float32)
    v = np.concatenate([mids, np.nextafter(mids, np.float32(9)), np.nextafter(mids, np.float32(-9))])
    v = np.concatenate([v, -v])
    top = 6.0 if fmt == qg.GEMM_NVFP4 else 7.9  # MXFP4: magnitudes between 6 and 8 saturate
    v = v[np.abs(v) <= top]
    b = R.BLOCK[fmt]
    x = np.zeros((1, R.ceil(len(v), b - 1) * b), dtype=np.float32)
    for i in range(x.shape[1] // b):
        part = v[i * (b - 1):(i + 1) * (b - 1)]
        x[0, i * b] = top
        x[0, i * b + 1:i * b + 1 + len(part)] = part
    x = torch.from_numpy(x).cuda()
    o, _ = quantize(h, x, fmt)
    packed, scales = expect(x, fmt)
    assert np.array_equal(o.scales.cpu().numpy(), R.tile(R.quantize(x.double().cpu().numpy(), fmt)[1], fill=0xAA))
    assert np.array_equal(o.codes.cpu().numpy(), packed)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
def test_special_values(h, fmt, dtype):
    big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    sub = float(torch.finfo(dtype).smallest_normal) / 4
    rows = [[0.0] * 32, [float("nan")] + [1.0] * 31, [1.0] * 31 + [float("inf")], [float("-inf")] + [2.0] * 31,
            [big] * 32, [-big, 1.0] + [0.0] * 30, [tiny] * 32, [sub] * 32, [-0.0] * 32, [sub, 1.0] * 16,
            [2.0 ** -9 * 6] * 32, [2.0 ** -10 * 6] * 32, [448.0 * 6] * 32, [449.0 * 6] * 32]
    x = torch.tensor(rows, dtype=torch.float64).to(dtype).cuda()
    o, _ = quantize(h, x, fmt)
    packed, scales = expect(x, fmt)
    assert np.array_equal(o.scales.cpu().numpy(), scales)
    assert np.array_equal(o.codes.cpu().numpy(), packed)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts", [[5], [3, 0, 4], [0, 0, 130, 1], [128, 1, 128], [1] * 70, [0] * 40 + [9] + [0] * 30])
def test_rows_by_expert(h, fmt, counts):
    x = values(sum(counts), 200, torch.bfloat16, seed=len(counts))
    o, off = quantize(h, x, fmt, counts=counts)
    packed, scales = expect(x, fmt, counts=counts)
    assert np.array_equal(o.scales.cpu().numpy(), scales) and np.array_equal(o.codes.cpu().numpy(), packed)
    out = torch.empty(x.shape, dtype=torch.float32, device="cuda")
    c, cl, s, sb = o.args()
    assert qg.gemm_mx_dequantize(h, fmt, 1.0, c, cl, s, sb, qg.ptr(out), qg.row_major(out), qg.ptr(off), len(counts),
                                 qg.current_stream()) == 0
    assert np.array_equal(out.double().cpu().numpy(), R.dequantize(*R.quantize(x.double().cpu().numpy(), fmt), fmt))


def test_rows_past_the_experts_are_left_out(h):
    x = values(20, 64, torch.bfloat16)
    o = qg.MxOperand(qg.GEMM_NVFP4, 20, 64, num_experts=2)
    o.codes.fill_(0xAA)
    off = torch.tensor([0, 3, 12], dtype=torch.int32, device="cuda")
    c, cl, s, sb = o.args()
    assert qg.gemm_mx_quantize(h, qg.GEMM_NVFP4, 1.0, qg.ptr(x), qg.row_major(x), c, cl, s, sb, qg.ptr(off), 2,
                               qg.current_stream()) == 0
    got = o.codes.cpu().numpy()
    assert np.array_equal(got[:12], R.pack(R.quantize(x[:12].double().cpu().numpy(), R.NVFP4)[0]))
    assert (got[12:] == 0xAA).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_several_matrices(h, fmt):
    x = torch.stack([values(130, 96, torch.float16, seed=i) for i in range(3)])
    o, _ = quantize(h, x, fmt)
    per = o.scales.numel() // 3
    for i in range(3):
        packed, scales = expect(x[i], fmt)
        assert np.array_equal(o.codes[i].cpu().numpy(), packed)
        assert np.array_equal(o.scales[i * per:(i + 1) * per].cpu().numpy(), scales)
    out = torch.empty(x.shape, dtype=torch.float32, device="cuda")
    c, cl, s, sb = o.args()
    assert qg.gemm_mx_dequantize(h, fmt, 1.0, c, cl, s, sb, qg.ptr(out), qg.row_major(out), None, 0,
                                 qg.current_stream()) == 0
    for i in range(3):
        want = R.dequantize(*R.quantize(x[i].double().cpu().numpy(), fmt), fmt)
        assert np.array_equal(out[i].double().cpu().numpy(), want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES + [torch.float8_e4m3fn])
@pytest.mark.parametrize("shape,pad", [((3, 33), 0), ((150, 512), 16), ((7, 1031), 1), ((1, 1), 0)])
def test_dequantize(h, fmt, dtype, shape, pad):
    rows, k = shape
    rng = np.random.default_rng(k)
    code, byte = R.random_operand(rng, rows, k, fmt)
    o = qg.MxOperand(fmt, rows, k)
    o.codes.copy_(torch.from_numpy(R.pack(code)))
    o.scales[:R.tile(byte).size].copy_(torch.from_numpy(R.tile(byte)))
    raw = dtype == torch.float8_e4m3fn
    g = 0.75 if fmt == qg.GEMM_NVFP4 else 1.0
    buf = torch.full((rows, k + pad), 3.0, dtype=torch.float32).to(dtype).cuda()
    out = buf[:, :k]
    c, cl, s, sb = o.args()
    rc = qg.gemm_mx_dequantize(h, fmt, g, c, cl, s, sb, qg.ptr(out), qg.row_major(out), None, 0, qg.current_stream())
    assert rc == 0, qg.gemm_status_string(rc)
    # code * scale * 0.75 has at most 8 significant bits: exact in every type
    want = R.VALUES[code] if raw else R.dequantize(code, byte, fmt, g)
    assert np.array_equal(out.to(torch.float64).cpu().numpy(), want)
    assert bool((buf[:, k:].float() == 3).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_dequantize_nan_scale(h, fmt):
    x = torch.ones(2, 64, device="cuda")
    x[1, 5] = float("nan")
    o, _ = quantize(h, x, fmt)
    out = torch.empty_like(x)
    c, cl, s, sb = o.args()
    assert qg.gemm_mx_dequantize(h, fmt, 1.0, c, cl, s, sb, qg.ptr(out), qg.row_major(out), None, 0,
                                 qg.current_stream()) == 0
    b = R.BLOCK[fmt]
    one = float(R.dequantize(*R.quantize(np.ones((1, b)), fmt), fmt)[0, 0])  # 1 as the format holds it
    assert bool(out[1, :b].isnan().all()) and bool((out[0] == one).all()) and bool((out[1, b:] == one).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("off", range(8))
def test_rows_that_start_anywhere(h, dtype, off):
    # odd row strides put every row at another distance from a 16-byte boundary;
    # what is read past a row must not matter, nothing past it may be written
    rows, k, ld = 33, 1091, 1101
    buf = torch.full((rows * ld + 8,), float("nan"), dtype=dtype, device="cuda")
    x = buf[off:off + rows * ld].view(rows, ld)[:, :k]
    x.copy_(values(rows, k, dtype, seed=off))
    o, _ = quantize(h, x, qg.GEMM_NVFP4)
    packed, scales = expect(x, qg.GEMM_NVFP4)
    assert np.array_equal(o.scales.cpu().numpy(), scales) and np.array_equal(o.codes.cpu().numpy(), packed)
    c, cl, s, sb = o.args()
    code, byte = R.quantize(x.double().cpu().numpy(), qg.GEMM_NVFP4)
    for out_t, want in ((dtype, R.dequantize(code, byte, qg.GEMM_NVFP4)), (torch.float8_e4m3fn, R.VALUES[code])):
        back = torch.full((rows * ld + 8,), 7.0, device="cuda").to(out_t)
        y = back[off:off + rows * ld].view(rows, ld)[:, :k]
        assert qg.gemm_mx_dequantize(h, qg.GEMM_NVFP4, 1.0, c, cl, s, sb, qg.ptr(y), qg.row_major(y), None, 0,
                                     qg.current_stream()) == 0
        # code * scale has at most 6 significant bits: exact in every type, but for
        # fp16's smallest values
        want_t = torch.from_numpy(want).to(out_t).double().numpy() if out_t == torch.float16 else want
        assert np.array_equal(y.double().cpu().numpy() if out_t != torch.float8_e4m3fn else y.float().double().cpu().numpy(), want_t)
        around = back.float().cpu().clone()
        around[off:off + rows * ld].view(rows, ld)[:, :k] = 7.0
        assert bool((around == 7.0).all())
