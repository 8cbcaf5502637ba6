"""GPU tests of the residual norm that quantises its result
(gemm_mx_norm_quantize) against numpy in 64 bits.

Tolerances.  A thread adds at most 64 squares one after another and the block
adds 5 + 16 more levels, all positive: the sum's relative error is at most
85 * 2^-24, half of that after the square root; with the reciprocal root's
2 ulp and three products a normed value is within DELTA = 4e-6.  The residual
then differs from its rounded exact value by DELTA * |scale u|, two fp32
roundings and one ulp of its type.  Codes and scales are a function of the
residual as stored, so they are checked from the residual that came back: the
scale byte must be that of a block maximum within DELTA, each code that of a
value within DELTA under that scale."""
import numpy as np
import pytest
import torch

import mx_ref as R
import oracle
import quantized_gemm_tcgen05_gb300 as qg
import synth

pytestmark = pytest.mark.gpu

DELTA = 4e-6
FORMATS = [qg.GEMM_NVFP4, qg.GEMM_MXFP4]
TD = {synth.F32: torch.float32, synth.F16: torch.float16, synth.BF16: torch.bfloat16}


@pytest.fixture(scope="module")
def h():
    h = qg.gemm_create()
    yield h
    qg.gemm_destroy(h)


def f64(t):
    return t.double().cpu().numpy()


def run(h, fmt, f, r, post=None, pre=None, gate=None, gate_ld=0, eps=1e-5, rs=0.7, g=1.0, out=None, wt=None):
    rows, cols = r.shape
    o = qg.MxOperand(fmt, rows, cols)
    o.codes.fill_(0xAA)
    o.scales.fill_(0xAA)
    n = qg.gemm_mx_norm_t(format=fmt, tensor_scale=g, eps=eps, residual_scale=rs)
    n.weight_type = wt if wt is not None else qg.row_major(r).type
    if post is not None:
        n.post_weight = qg.ptr(post)
    if pre is not None:
        n.pre_weight = qg.ptr(pre)
    if gate is not None:
        n.gate, n.gate_type, n.gate_ld = qg.ptr(gate), qg._dtype_code(gate.dtype), gate_ld
    if out is None and f is not None:
        out = torch.full((rows, cols), float("nan"), dtype=r.dtype, device="cuda")
    c, cl, s, sb = o.args()
    rc = qg.gemm_mx_norm_quantize(h, n, qg.ptr(f), None if f is None else qg.row_major(f), qg.ptr(r), qg.row_major(r),
                                  qg.ptr(out), None if out is None else qg.row_major(out), c, cl, s, sb,
                                  qg.current_stream())
    assert rc == 0, qg.gemm_status_string(rc)
    torch.cuda.synchronize()
    return out, o


def check_residual(out, f, r, post, gate, eps, rs, dt):
    u = f64(f)
    if post is not None:
        u = u / np.sqrt((u * u).mean(-1, keepdims=True) + eps) * f64(post)
    if gate is not None:
        u = u * f64(gate)
    want = f64(r) + rs * u
    tol = DELTA * np.abs(rs * u) + 2.0 ** -22 * np.abs(want) + 1e-30
    if dt != synth.F32:
        tol = tol + oracle.ulp(dt, want)
    assert (np.abs(f64(out) - want) <= tol).all()


def check_codes(o, resid, pre, eps, fmt, g=1.0):
    v = f64(resid)
    rows, k = v.shape
    y = v / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    if pre is not None:
        y = y * f64(pre)
    b = R.BLOCK[fmt]
    nb = R.ceil(k, b)
    flat = o.scales.cpu().numpy()
    atoms = R.ceil(nb, 4)
    got = flat[R.scale_at(np.arange(rows)[:, None], np.arange(atoms * 4)[None], atoms)]
    assert (got[:, nb:] == 0).all()
    got = got[:, :nb]
    lo, hi = R.quantize(y * (1 - DELTA), fmt, g)[1], R.quantize(y * (1 + DELTA), fmt, g)[1]
    assert ((got >= np.minimum(lo, hi)) & (got <= np.maximum(lo, hi))).all()
    s = np.repeat(R.scale_values(got, fmt) * g, b, axis=1)[:, :k]
    with np.errstate(all="ignore"):
        w = np.where(s > 0, y / s, 0.0)
    code = R.unpack(o.codes.cpu().numpy(), k)
    mag = np.abs(w)
    a, z = R.nearest(R.MAG, mag * (1 - DELTA)), R.nearest(R.MAG, mag * (1 + DELTA))
    m = code & 7
    assert ((m >= a) & (m <= z)).all()
    assert ((code >> 3 == np.signbit(w)) | (m == 0)).all()
    assert (o.codes.cpu().numpy()[:, R.ceil(k, 2):] == 0xAA).all()


def data(rows, cols, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    t = torch.randn(rows, cols + pad, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))
    return t.to(dtype).cuda()[:, :cols]


SHAPES = [(1, 1), (1, 4096), (3, 33), (2, 16), (130, 257), (7, 1031), (64, 4096), (5, 4112), (3, 8200), (2, 14336), (2, 16400), (1, 32768)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dt", [synth.F32, synth.F16, synth.BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_all_parts(h, fmt, dt, shape):
    rows, cols = shape
    f, r = data(rows, cols, TD[dt], 1), data(rows, cols, TD[dt], 2)
    post, pre = data(1, cols, TD[dt], 3)[0], data(1, cols, TD[dt], 4)[0]
    gate = torch.tanh(data(rows, cols, torch.float32, 5)).to(TD[dt])
    out, o = run(h, fmt, f, r, post, pre, gate, gate_ld=cols)
    check_residual(out, f, r, post, gate, 1e-5, 0.7, dt)
    check_codes(o, out, pre, 1e-5, fmt)
    again, o2 = run(h, fmt, f, r, post, pre, gate, gate_ld=cols)
    assert torch.equal(out, again) and torch.equal(o.codes, o2.codes) and torch.equal(o.scales, o2.scales)


@pytest.mark.parametrize("post,pre,gate", [(0, 0, 0), (1, 0, 0), (0, 1, 1), (0, 0, 2), (1, 1, 1)])
def test_parts_left_out(h, post, pre, gate):
    rows, cols, fmt = 19, 600, qg.GEMM_NVFP4
    f, r = data(rows, cols, torch.bfloat16, 1), data(rows, cols, torch.bfloat16, 2)
    pw = data(1, cols, torch.bfloat16, 3)[0] if post else None
    nw = data(1, cols, torch.bfloat16, 4)[0] if pre else None
    gt = [None, data(1, cols, torch.float32, 5)[0], data(rows, cols, torch.float16, 6, pad=40)][gate]
    out, o = run(h, fmt, f, r, pw, nw, gt, gate_ld=cols + 40 if gate == 2 else 0, rs=-1.25, eps=1e-3, g=0.25)
    check_residual(out, f, r, pw, gt, 1e-3, -1.25, synth.BF16)
    check_codes(o, out, nw, 1e-3, fmt, g=0.25)


@pytest.mark.parametrize("fmt", FORMATS)
def test_first_layer_has_no_block_before_it(h, fmt):
    r, pre = data(9, 512, torch.float16, 1), data(1, 512, torch.float32, 2)[0]
    _, o = run(h, fmt, None, r, pre=pre, wt=qg.GEMM_F32)
    check_codes(o, r, pre, 1e-5, fmt)
    out = torch.empty(9, 512, dtype=torch.float16, device="cuda")
    run(h, fmt, None, r, pre=pre, wt=qg.GEMM_F32, out=out)
    assert torch.equal(out, r)


@pytest.mark.parametrize("which", ["r", "f"])
def test_in_place(h, which):
    f, r = data(33, 1000, torch.bfloat16, 1), data(33, 1000, torch.bfloat16, 2)
    w = data(1, 1000, torch.bfloat16, 3)[0]
    want, o = run(h, qg.GEMM_NVFP4, f, r, post=w, pre=w)
    f2, r2 = f.clone(), r.clone()
    got, o2 = run(h, qg.GEMM_NVFP4, f2, r2, post=w, pre=w, out=r2 if which == "r" else f2)
    assert torch.equal(got, want) and torch.equal(o.codes, o2.codes) and torch.equal(o.scales, o2.scales)


def test_strided_rows_and_neighbours(h):
    rows, cols = 20, 333
    f, r = data(rows, cols, torch.float16, 1, pad=11), data(rows, cols, torch.float16, 2, pad=3)
    buf = torch.full((rows, cols + 6), 2.0, dtype=torch.float16, device="cuda")
    pre = data(1, cols + 1, torch.float16, 3)[0, 1:]  # element-aligned weights
    out, o = run(h, qg.GEMM_MXFP4, f, r, pre=pre, out=buf[:, :cols])
    check_residual(out, f, r, None, None, 1e-5, 0.7, synth.F16)
    check_codes(o, out, pre, 1e-5, qg.GEMM_MXFP4)
    assert bool((buf[:, cols:] == 2).all())


def test_zero_and_nan_rows(h):
    f, r = data(3, 256, torch.float32, 1), data(3, 256, torch.float32, 2)
    f[0], r[0] = 0, 0
    f[1, 7] = float("nan")
    out, o = run(h, qg.GEMM_NVFP4, f, r)
    assert bool((out[0] == 0).all()) and int((o.codes[0] & 0x77).max()) == 0
    # one NaN in the residual makes every normed value of its row NaN, no other row's
    s = o.scales.cpu().numpy()
    nan = [(s[R.scale_at(np.full(16, i), np.arange(16), 4)] == 0x7F).all() for i in range(3)]
    assert nan == [False, True, False]
    check_codes_rows = torch.isnan(out).any(-1).cpu().tolist()
    assert check_codes_rows == [False, True, False]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts,extra", [([3, 0, 130, 1], 0), ([0, 5], 2), ([1] * 40, 0)])
def test_rows_by_expert(h, fmt, counts, extra):
    # the same row by row, scales on the experts' own atom rows
    rows, cols = sum(counts) + extra, 272
    f, r = data(rows, cols, torch.bfloat16, 1), data(rows, cols, torch.bfloat16, 2)
    pre = data(1, cols, torch.bfloat16, 3)[0]
    want, o = run(h, fmt, f, r, pre=pre)
    off = np.concatenate([[0], np.cumsum(counts)])
    offd = torch.from_numpy(off.astype(np.int32)).cuda()
    e = qg.MxOperand(fmt, rows, cols, num_experts=len(counts))
    e.codes.fill_(0xAA)
    n = qg.gemm_mx_norm_t(format=fmt, tensor_scale=1.0, eps=1e-5, residual_scale=0.7, pre_weight=qg.ptr(pre),
                          weight_type=qg.GEMM_BF16, expert_offsets=qg.ptr(offd), num_experts=len(counts))
    out = torch.empty_like(want)
    lay = qg.row_major(r)
    rc = qg.gemm_mx_norm_quantize(h, n, qg.ptr(f), qg.row_major(f), qg.ptr(r), lay, qg.ptr(out), qg.row_major(out), *e.args(),
                                  qg.current_stream())
    assert rc == 0
    held = sum(counts)
    assert torch.equal(out, want) and torch.equal(e.codes[:held], o.codes[:held])
    assert bool((e.codes[held:] == 0xAA).all())
    nb = R.ceil(cols, R.BLOCK[fmt])
    atoms, j = R.ceil(nb, 4), np.arange(nb)[None]
    a = e.scales.cpu().numpy()[R.scale_at(R.expert_rows(off)[:, None], j, atoms)]
    b = o.scales.cpu().numpy()[R.scale_at(np.arange(held)[:, None], j, atoms)]
    assert np.array_equal(a, b)


@pytest.mark.parametrize("dt", [synth.F32, synth.F16, synth.BF16])
@pytest.mark.parametrize("off", [0, 1, 2, 3, 5, 7])
@pytest.mark.parametrize("cols", [1091, 5003])
def test_rows_that_start_anywhere(h, dt, off, cols):
    rows, ld = 9, cols + 10

    def odd(seed):
        buf = torch.full((rows * ld + 8,), float("nan"), dtype=TD[dt], device="cuda")
        t = buf[off:off + rows * ld].view(rows, ld)[:, :cols]
        t.copy_(data(rows, cols, TD[dt], seed))
        return t

    f, r, gate = odd(1), odd(2), odd(3)
    post, pre = odd(4)[0], odd(5)[0]
    back = torch.full((rows * ld + 8,), 7.0, dtype=TD[dt], device="cuda")
    out, o = run(h, qg.GEMM_NVFP4, f, r, post, pre, gate, gate_ld=ld, out=back[off:off + rows * ld].view(rows, ld)[:, :cols])
    check_residual(out, f, r, post, gate, 1e-5, 0.7, dt)
    check_codes(o, out, pre, 1e-5, qg.GEMM_NVFP4)
    # the same bits as from rows that start on 16-byte boundaries
    even = lambda t: t.contiguous() if cols % 8 == 0 else torch.cat([t, t[..., :(-cols) % 16]], -1)[..., :cols]  # noqa: E731
    same, o2 = run(h, qg.GEMM_NVFP4, even(f), even(r), post.clone(), pre.clone(), even(gate), gate_ld=even(gate).stride(0))
    assert torch.equal(out, same) and torch.equal(o.codes, o2.codes) and torch.equal(o.scales, o2.scales)
    around = back.float().cpu().clone()
    around[off:off + rows * ld].view(rows, ld)[:, :cols] = 7.0
    assert bool((around == 7.0).all())
