"""GPU parity of the 4-bit microscaled products (gemm_run_mx,
gemm_run_mx_grouped) against numpy in 64 bits: operand and scale placement
bit by bit, ragged sizes in all three dimensions, output types, epilogues,
strides, K slices, experts with and without rows, NaN scales, and that
nothing outside D is written."""
import numpy as np
import pytest
import torch

import mx_ref as R
import oracle
import quantized_gemm_tcgen05_gb300 as qg
import synth

pytestmark = pytest.mark.gpu

TD = {synth.F32: torch.float32, synth.F16: torch.float16, synth.BF16: torch.bfloat16}
FORMATS = [qg.GEMM_NVFP4, qg.GEMM_MXFP4]
OUTS = [synth.F32, synth.F16, synth.BF16]


@pytest.fixture(scope="module")
def h():
    h = qg.gemm_create()
    yield h
    qg.gemm_destroy(h)


@pytest.fixture(params=["", "mx_bn64", "mx_bn128", "mx2_bn256"])
def kernel(request, monkeypatch):
    """The automatic choice, then each kernel pinned."""
    if request.param:
        monkeypatch.setenv("GEMM_FORCE_KERNEL", request.param)
    return request.param


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def tol(ref, bound, d):
    t = 1e-5 * bound + 1e-6
    return t if d == synth.F32 else t + oracle.ulp(d, ref)


class Operand:
    """Codes and scales on the host (values in 64 bits) and on the device."""

    def __init__(self, rng, rows, k, fmt, code=None, byte=None, ld=None, row=None, tiles=None):
        c, b = R.random_operand(rng, rows, k, fmt)
        self.code = c if code is None else code
        self.byte = b if byte is None else byte
        self.values = R.dequantize(self.code, self.byte, fmt)
        self.k = k
        self.packed = dev(R.pack(self.code, ld))
        # scale rows that hold nothing are NaN bytes: no result may depend on them
        self.scales = dev(R.tile(self.byte, row, tiles, fill=0x7F if fmt == qg.GEMM_NVFP4 else 0xFF))


def product(h, a, b, fmt, d, alpha=1.0, beta=0.0, c=None, op=None, out=None, ldd=None):
    m, n = a.code.shape[0], b.code.shape[0]
    if out is None:
        out = torch.full((m, n if ldd is None else ldd), float("nan"), dtype=TD[d], device="cuda")
    op = op or qg.gemm_op_t()
    rc = qg.gemm_run_mx(h, op, fmt, alpha, qg.ptr(a.packed), qg.mx_layout(a.packed, a.k), qg.ptr(a.scales),
                        a.scales.numel(), qg.ptr(b.packed), qg.mx_layout_b(b.packed, b.k), qg.ptr(b.scales),
                        b.scales.numel(), beta, qg.ptr(c), None if c is None else qg.layout(d, 0, m, n, c.stride(0)),
                        qg.ptr(out), qg.layout(d, 0, m, n, out.stride(0)), qg.current_stream())
    assert rc == 0, qg.gemm_status_string(rc)
    assert qg.gemm_device_status(h, qg.current_stream()) == 0
    return out


def check(got, ref, bound, d, what=""):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - ref) <= tol(ref, bound, d))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, first {np.argwhere(bad)[0]}: " \
                          f"{got[tuple(np.argwhere(bad)[0])]} want {ref[tuple(np.argwhere(bad)[0])]}"


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("splits", [0, 1, 2])
def test_one_hot_placement(h, monkeypatch, fmt, splits):
    # A has one code per row (1.0, scale 1) at k = 37 i % K: D[i][j] is exactly
    # B's value there, so a misplaced code, scale row or scale column shows
    if splits == 0:
        monkeypatch.setenv("GEMM_FORCE_KERNEL", "mx2_bn256")
    m, n, k = 256, 320, 1088
    rng = np.random.default_rng(5)
    code = np.zeros((m, k), np.uint8)
    hot = 37 * np.arange(m) % k
    code[np.arange(m), hot] = 2
    one = 0x38 if fmt == qg.GEMM_NVFP4 else 127
    a = Operand(rng, m, k, fmt, code=code, byte=np.full((m, R.ceil(k, R.BLOCK[fmt])), one, np.uint8))
    b = Operand(rng, n, k, fmt)
    op = qg.gemm_op_t(splitk=splits)
    got = product(h, a, b, fmt, synth.F32, op=op).double().cpu().numpy()
    assert np.array_equal(got, b.values[:, hot].T)
    # and the other way round: B one-hot, A random
    got = product(h, b, a, fmt, synth.F32, op=op).double().cpu().numpy()
    assert np.array_equal(got, b.values[:, hot])


SHAPES = [(1, 1, 1), (1, 4096, 512), (3, 130, 95), (17, 64, 256), (64, 1000, 4096), (127, 129, 33), (128, 128, 257),
          (129, 257, 700), (200, 328, 1031), (300, 1002, 2080), (520, 700, 31), (1, 8, 14336), (256, 512, 64),
          (640, 1280, 768), (1000, 2056, 1280), (257, 300, 1600)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d", OUTS)
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(h, kernel, fmt, d, shape):
    m, n, k = shape
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    a, b = Operand(rng, m, k, fmt), Operand(rng, n, k, fmt)
    alpha = 0.25 if d == synth.F16 else 1.5
    ref, bound = alpha * a.values @ b.values.T, abs(alpha) * np.abs(a.values) @ np.abs(b.values).T
    if d == synth.F16:  # within the type's range
        alpha /= 64
        ref, bound = ref / 64, bound / 64
    check(product(h, a, b, fmt, d, alpha=alpha), ref, bound, d, f"{shape} {qg.gemm_last_choice(h)}")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("splits", [1, 2, 4, 8])
@pytest.mark.parametrize("shape", [(5, 192, 2300), (130, 200, 4096)])
def test_k_slices(h, fmt, splits, shape):
    m, n, k = shape
    rng = np.random.default_rng(splits)
    a, b = Operand(rng, m, k, fmt), Operand(rng, n, k, fmt)
    op = qg.gemm_op_t(splitk=splits)
    ref, bound = a.values @ b.values.T, np.abs(a.values) @ np.abs(b.values).T
    got = product(h, a, b, fmt, synth.F32, op=op)
    check(got, ref, bound, synth.F32, qg.gemm_last_choice(h))
    for _ in range(3):  # the same bits every time
        assert torch.equal(got, product(h, a, b, fmt, synth.F32, op=op))


@pytest.mark.parametrize("d", OUTS)
@pytest.mark.parametrize("act", ["", "bias", "relu", "gelu"])
@pytest.mark.parametrize("shape,splits,pin", [((70, 264, 600), 1, ""), ((70, 264, 600), 2, ""), ((300, 517, 512), 1, ""),
                                              ((600, 1100, 512), 1, "mx2_bn256"), ((260, 520, 300), 0, "mx2_bn256")])
def test_epilogue(h, monkeypatch, d, act, shape, splits, pin):
    if pin:
        monkeypatch.setenv("GEMM_FORCE_KERNEL", pin)
    fmt = qg.GEMM_NVFP4
    m, n, k = shape
    rng = np.random.default_rng(11)
    a, b = Operand(rng, m, k, fmt), Operand(rng, n, k, fmt)
    c = torch.randn(m, n, generator=torch.Generator().manual_seed(1)).to(TD[d]).cuda()
    op = qg.gemm_op_t(splitk=splits)
    alpha, beta = 2.0 ** -7, 0.5
    x = alpha * a.values @ b.values.T + beta * c.double().cpu().numpy()
    bound = alpha * np.abs(a.values) @ np.abs(b.values).T + beta * np.abs(c.double().cpu().numpy())
    if act:
        bias = torch.randn(n, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
        op.epilogue, op.bias, op.bias_type = qg.GEMM_EPILOGUE_BIAS, qg.ptr(bias), qg.GEMM_BF16
        bv = bias.double().cpu().numpy()
        x, bound = x + bv, bound + np.abs(bv)
    if act == "relu":
        op.epilogue |= qg.GEMM_EPILOGUE_RELU
        x = np.maximum(x, 0.0)
    if act == "gelu":
        op.epilogue |= qg.GEMM_EPILOGUE_GELU
        t = torch.from_numpy(x)
        x, bound = (0.5 * t * (1 + torch.erf(t / 2 ** 0.5))).numpy(), 1.129 * bound
    check(product(h, a, b, fmt, d, alpha=alpha, beta=beta, c=c, op=op), x, bound, d, act)
    # in place: C is D
    out = c.clone()
    assert torch.equal(product(h, a, b, fmt, d, alpha=alpha, beta=beta, c=out, op=op, out=out),
                       product(h, a, b, fmt, d, alpha=alpha, beta=beta, c=c, op=op))


@pytest.mark.parametrize("d", OUTS)
@pytest.mark.parametrize("ldd", [200, 208, 217, 256])
def test_strides_and_nothing_else_written(h, kernel, d, ldd):
    fmt = qg.GEMM_MXFP4
    m, n, k = 150, 199, 320
    rng = np.random.default_rng(ldd)
    a, b = Operand(rng, m, k, fmt, ld=416), Operand(rng, n, k, fmt, ld=352)
    buf = torch.full((m + 2, ldd), 7.0, dtype=TD[d], device="cuda")
    out = buf[1:m + 1]
    product(h, a, b, fmt, d, alpha=2.0 ** -6, out=out)
    ref, bound = 2.0 ** -6 * a.values @ b.values.T, 2.0 ** -6 * np.abs(a.values) @ np.abs(b.values).T
    check(out[:, :n], ref, bound, d)
    assert bool((buf[0] == 7).all()) and bool((buf[-1] == 7).all()) and bool((buf[:, n:] == 7).all())


def test_element_aligned_output(h, kernel):
    # D starts one element into its buffer: no vector access may be used
    fmt, m, n, k = qg.GEMM_NVFP4, 66, 128, 128
    rng = np.random.default_rng(1)
    a, b = Operand(rng, m, k, fmt), Operand(rng, n, k, fmt)
    buf = torch.full((m * n + 8,), 3.0, dtype=torch.bfloat16, device="cuda")
    out = buf[1:1 + m * n].view(m, n)
    product(h, a, b, fmt, synth.BF16, out=out)
    check(out, a.values @ b.values.T, np.abs(a.values) @ np.abs(b.values).T, synth.BF16)
    assert float(buf[0]) == 3 and bool((buf[1 + m * n:] == 3).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_nan_scale_reaches_its_row_and_column_only(h, kernel, fmt):
    m, n, k = 40, 140, 512
    rng = np.random.default_rng(3)
    a, b = Operand(rng, m, k, fmt), Operand(rng, n, k, fmt)
    nan = 0x7F if fmt == qg.GEMM_NVFP4 else 0xFF
    a.byte[7, 2] = nan
    b.byte[133, 0] = nan
    a = Operand(rng, m, k, fmt, code=a.code, byte=a.byte)
    b = Operand(rng, n, k, fmt, code=b.code, byte=b.byte)
    got = product(h, a, b, fmt, synth.F32).cpu().numpy()
    want = np.zeros((m, n), bool)
    want[7], want[:, 133] = True, True
    assert np.array_equal(np.isnan(got), want)


@pytest.mark.parametrize("beta,act", [(0.0, 0), (2.0, 0), (2.0, qg.GEMM_EPILOGUE_RELU)])
def test_no_k(h, beta, act):
    m, n = 5, 7
    c = torch.randn(m, n, device="cuda")
    out = torch.full((m, n), 9.0, device="cuda")
    e = torch.zeros(8, 16, dtype=torch.uint8, device="cuda")
    op = qg.gemm_op_t(epilogue=act)
    rc = qg.gemm_run_mx(h, op, qg.GEMM_NVFP4, 1.0, qg.ptr(e), qg.layout(7, 0, m, 0, 32), qg.ptr(e), 0, qg.ptr(e),
                        qg.layout(7, 1, 0, n, 32), qg.ptr(e), 0, beta, qg.ptr(c), qg.row_major(c), qg.ptr(out),
                        qg.row_major(out), qg.current_stream())
    assert rc == 0
    want = beta * c
    assert torch.equal(out, torch.relu(want) if act else want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_tiles_per_program(h, fmt):
    # every cluster of the CTA-pair kernel runs several tiles, ragged ones last
    m, n, k = 2600, 5000, 320
    rng = np.random.default_rng(21)
    a, b = Operand(rng, m, k, fmt), Operand(rng, n, k, fmt)
    got = product(h, a, b, fmt, synth.BF16, alpha=0.5)
    assert qg.gemm_last_choice(h).startswith("mx2_")
    check(got, 0.5 * a.values @ b.values.T, 0.5 * np.abs(a.values) @ np.abs(b.values).T, synth.BF16)
    assert torch.equal(got, product(h, a, b, fmt, synth.BF16, alpha=0.5))


# ---- grouped -----------------------------------------------------------------

def grouped(h, counts, n, k, fmt, d, seed, alpha=1.0, with_expert_alpha=True, beta=0.0, extra=0, op=None):
    rng = np.random.default_rng(seed)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    rows, E = int(off[-1]) + extra, len(counts)
    held = R.expert_rows(off)
    a = Operand(rng, rows - extra, k, fmt, row=held, tiles=rows // 128 + E)
    if extra:  # rows past the last expert's: no codes of interest, no result
        a.packed = torch.cat([a.packed, torch.zeros(extra, a.packed.shape[1], dtype=torch.uint8, device="cuda")])
    w = [Operand(rng, n, k, fmt) for _ in range(E)]
    packed, scales = torch.stack([x.packed for x in w]), torch.cat([x.scales for x in w])
    ea = torch.rand(E, generator=torch.Generator().manual_seed(seed)).cuda() + 0.5
    offd = dev(off.astype(np.int32))
    out = torch.full((rows, n), 5.0, dtype=TD[d], device="cuda")
    c = torch.randn(rows, n, generator=torch.Generator().manual_seed(seed)).to(TD[d]).cuda() if beta else None
    rc = qg.gemm_run_mx_grouped(h, op or qg.gemm_op_t(), fmt, alpha, qg.ptr(ea) if with_expert_alpha else None,
                                qg.ptr(a.packed), qg.mx_layout(a.packed, k), qg.ptr(a.scales), a.scales.numel(),
                                qg.ptr(packed), qg.mx_layout_b(packed, k), qg.ptr(scales), scales.numel(), beta,
                                qg.ptr(c), None if c is None else qg.row_major(c), qg.ptr(out), qg.row_major(out),
                                qg.ptr(offd), E, qg.current_stream())
    assert rc == 0, qg.gemm_status_string(rc)
    assert qg.gemm_device_status(h, qg.current_stream()) == 0
    ref, bound = np.zeros((rows, n)), np.zeros((rows, n))
    for e in range(E):
        s = slice(off[e], off[e + 1])
        f = alpha * (float(ea[e]) if with_expert_alpha else 1.0)
        ref[s], bound[s] = f * a.values[s] @ w[e].values.T, f * np.abs(a.values[s]) @ np.abs(w[e].values).T
    if beta:
        ref += beta * c.double().cpu().numpy()
        bound += beta * np.abs(c.double().cpu().numpy())
    last = rows - extra
    check(out[:last], ref[:last], bound[:last], d, f"{counts} {qg.gemm_last_choice(h)}")
    if extra:
        assert bool((out[last:] == 5).all())


COUNTS = [[1], [5, 0, 3], [0, 0, 0, 130], [128, 128, 1], [127, 129, 0, 256, 2], [0, 700, 0], [1] * 40,
          [0] * 33 + [7] + [0] * 30 + [2]]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts", COUNTS, ids=[str(i) for i in range(len(COUNTS))])
@pytest.mark.parametrize("n,k", [(192, 512), (137, 97)])
def test_grouped(h, kernel, fmt, counts, n, k):
    grouped(h, counts, n, k, fmt, synth.BF16, seed=len(counts) + n, alpha=0.125)


@pytest.mark.parametrize("d", OUTS)
def test_grouped_types_c_and_rows_past_the_experts(h, kernel, d):
    grouped(h, [200, 0, 57, 300], 300, 640, qg.GEMM_NVFP4, d, seed=4, alpha=2.0 ** -8, beta=0.5)
    grouped(h, [20, 0, 57], 128, 1500, qg.GEMM_MXFP4, d, seed=5, alpha=2.0 ** -8, with_expert_alpha=False, extra=9)


def test_offsets_past_the_rows_write_nothing_beyond_them(h, kernel):
    # offsets that promise more rows than A and D have: the rows there are come
    # out right, and nothing after them is touched
    fmt, n, k, have = qg.GEMM_NVFP4, 128, 256, 150
    rng = np.random.default_rng(9)
    off = np.array([0, 40, 400])
    held = R.expert_rows([0, 40, have])
    a = Operand(rng, have, k, fmt, row=held, tiles=have // 128 + 2)
    w = [Operand(rng, n, k, fmt) for _ in range(2)]
    packed, scales = torch.stack([x.packed for x in w]), torch.cat([x.scales for x in w])
    offd = dev(off.astype(np.int32))
    buf = torch.full((450, n), 5.0, device="cuda")
    rc = qg.gemm_run_mx_grouped(h, qg.gemm_op_t(), fmt, 1.0, None, qg.ptr(a.packed), qg.mx_layout(a.packed, k),
                                qg.ptr(a.scales), a.scales.numel(), qg.ptr(packed), qg.mx_layout_b(packed, k),
                                qg.ptr(scales), scales.numel(), 0.0, None, None, qg.ptr(buf),
                                qg.layout(synth.F32, 0, have, n, n), qg.ptr(offd), 2, qg.current_stream())
    assert rc == 0
    for e, s in ((0, slice(0, 40)), (1, slice(40, have))):
        check(buf[s], a.values[s] @ w[e].values.T, np.abs(a.values[s]) @ np.abs(w[e].values).T, synth.F32)
    assert bool((buf[have:] == 5).all())


@pytest.mark.parametrize("splits", [1, 2, 4])
def test_grouped_k_slices(h, splits):
    grouped(h, [3, 150, 0, 20], 256, 2048, qg.GEMM_NVFP4, synth.F32, seed=6, op=qg.gemm_op_t(splitk=splits))


def test_grouped_no_rows_at_all(h, kernel):
    grouped(h, [0, 0], 64, 64, qg.GEMM_NVFP4, synth.BF16, seed=7, extra=4)


@pytest.mark.parametrize("pin", ["", "mx2_bn256"])
@pytest.mark.parametrize("counts", [[1756, 764, 470, 333, 254, 204, 170, 145], [600, 0, 1, 255, 257, 512]])
def test_grouped_prompt(h, monkeypatch, counts, pin):
    if pin:
        monkeypatch.setenv("GEMM_FORCE_KERNEL", pin)
    grouped(h, counts, 1280, 1024, qg.GEMM_NVFP4, synth.BF16, seed=8, alpha=0.125)


# ---- streams, graphs -----------------------------------------------------------

def test_other_stream_and_graph(h):
    fmt, m, n, k = qg.GEMM_NVFP4, 96, 256, 1024
    rng = np.random.default_rng(2)
    a, b = Operand(rng, m, k, fmt), Operand(rng, n, k, fmt)
    want = product(h, a, b, fmt, synth.BF16)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        assert torch.equal(product(h, a, b, fmt, synth.BF16), want)
    out = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            rc = qg.gemm_run_mx(h, qg.gemm_op_t(), fmt, 1.0, qg.ptr(a.packed), qg.mx_layout(a.packed, k),
                                qg.ptr(a.scales), a.scales.numel(), qg.ptr(b.packed), qg.mx_layout_b(b.packed, k),
                                qg.ptr(b.scales), b.scales.numel(), 0.0, None, None, qg.ptr(out), qg.row_major(out),
                                qg.current_stream())
            assert rc == 0
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
