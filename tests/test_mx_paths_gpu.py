"""GPU tests of forms that the sizes of the other tests do not reach: the packed
epilogue with bias, ReLU and GELU in the kernels that have it, dense and by
expert, and the residual norm's walk over many rows, in place, by expert and
on rows that start anywhere.  Tolerances are those of test_mx_gemm_gpu.py and
test_mx_norm_gpu.py."""
import numpy as np
import pytest
import torch

import mx_ref as R
import quantized_gemm_tcgen05_gb300 as qg
import synth
import test_mx_gemm_gpu as G
import test_mx_norm_gpu as N

pytestmark = pytest.mark.gpu

ACTS = {"bias": 1, "relu": 1 | qg.GEMM_EPILOGUE_RELU, "gelu": 1 | qg.GEMM_EPILOGUE_GELU}


@pytest.fixture(scope="module")
def h():
    h = qg.gemm_create()
    yield h
    qg.gemm_destroy(h)


def activated(x, bound, act, bias):
    b = bias.double().cpu().numpy()
    x, bound = x + b, bound + np.abs(b)
    if act == "relu":
        return np.maximum(x, 0.0), bound
    if act == "gelu":
        t = torch.from_numpy(x)
        return (t * 0.5 * torch.special.erfc(-t / 2 ** 0.5)).numpy(), 1.129 * bound
    return x, bound


# ---- epilogues without C ---------------------------------------------------------

@pytest.mark.parametrize("d", [synth.BF16, synth.F16])
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("bias_type", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pin", ["mx_bn64", "mx_bn128", "mx2_bn256"])
@pytest.mark.parametrize("shape", [(300, 640, 520), (129, 1000, 256)])  # whole and ragged last columns
def test_dense(h, monkeypatch, pin, bias_type, act, d, shape):
    monkeypatch.setenv("GEMM_FORCE_KERNEL", pin)
    m, n, k = shape
    fmt, rng, alpha = qg.GEMM_NVFP4, np.random.default_rng(n), 2.0 ** -7
    a, b = G.Operand(rng, m, k, fmt), G.Operand(rng, n, k, fmt)
    bias = (2 * torch.randn(n, generator=torch.Generator().manual_seed(2))).to(bias_type).cuda()
    op = qg.gemm_op_t(epilogue=ACTS[act], bias=qg.ptr(bias), bias_type=qg._dtype_code(bias_type))
    out = torch.full((m, R.ceil(n, 16) * 16), 3.0, dtype=G.TD[d], device="cuda")
    G.product(h, a, b, fmt, d, alpha=alpha, op=op, out=out)
    x, bound = activated(alpha * a.values @ b.values.T, alpha * np.abs(a.values) @ np.abs(b.values).T, act, bias)
    G.check(out[:, :n], x, bound, d, f"{act} {qg.gemm_last_choice(h)}")
    assert bool((out[:, n:] == 3).all())


@pytest.mark.parametrize("d", [synth.BF16, synth.F16])
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("pin", ["mx_bn64", "mx_bn128", "mx2_bn256"])
def test_grouped(h, monkeypatch, pin, act, d):
    monkeypatch.setenv("GEMM_FORCE_KERNEL", pin)
    counts, n, k, fmt, alpha = [130, 0, 300, 7], 512, 512, qg.GEMM_MXFP4, 2.0 ** -6
    rng, E = np.random.default_rng(3), len(counts)
    off = np.concatenate([[0], np.cumsum(counts)])
    rows = int(off[-1])
    a = G.Operand(rng, rows, k, fmt, row=R.expert_rows(off), tiles=rows // 128 + E)
    w = [G.Operand(rng, n, k, fmt) for _ in range(E)]
    packed, scales = torch.stack([x.packed for x in w]), torch.cat([x.scales for x in w])
    bias = torch.randn(n, generator=torch.Generator().manual_seed(2)).cuda()
    ea = torch.rand(E, generator=torch.Generator().manual_seed(4)).cuda() + 0.5
    op = qg.gemm_op_t(epilogue=ACTS[act], bias=qg.ptr(bias), bias_type=qg.GEMM_F32)
    offd = G.dev(off.astype(np.int32))
    out = torch.full((rows, n), float("nan"), dtype=G.TD[d], device="cuda")
    rc = qg.gemm_run_mx_grouped(h, op, fmt, alpha, qg.ptr(ea), qg.ptr(a.packed), qg.mx_layout(a.packed, k), qg.ptr(a.scales),
                                a.scales.numel(), qg.ptr(packed), qg.mx_layout_b(packed, k), qg.ptr(scales),
                                scales.numel(), 0.0, None, None, qg.ptr(out), qg.row_major(out),
                                qg.ptr(offd), E, qg.current_stream())
    assert rc == 0 and qg.gemm_device_status(h, qg.current_stream()) == 0
    for e in range(E):
        s, f = slice(off[e], off[e + 1]), alpha * float(ea[e])
        x, bound = activated(f * a.values[s] @ w[e].values.T, f * np.abs(a.values[s]) @ np.abs(w[e].values).T, act, bias)
        G.check(out[s], x, bound, d, f"{act} {qg.gemm_last_choice(h)}")


# ---- the residual norm over more rows than blocks ---------------------------------

ROWS, COLS = 1500, 4096  # three blocks an SM walk three or four rows each


def many(dtype, seed):
    return N.data(ROWS, COLS, dtype, seed)


@pytest.mark.parametrize("dt", [synth.F16, synth.BF16])
@pytest.mark.parametrize("post,gate", [(True, True), (False, False)])
def test_norm_walks_many_rows(h, dt, post, gate):
    # bit by bit what calls of few rows give, whose blocks take one row each
    td, fmt = N.TD[dt], qg.GEMM_NVFP4
    f, r = many(td, 1), many(td, 2)
    pw = N.data(1, COLS, td, 3)[0] if post else None
    nw = N.data(1, COLS, td, 4)[0]
    gt = torch.tanh(N.data(ROWS, COLS, torch.float32, 5)).to(td) if gate else None
    out, o = N.run(h, fmt, f, r, pw, nw, gt, gate_ld=COLS if gate else 0)
    N.check_residual(out, f, r, pw, gt, 1e-5, 0.7, dt)
    atoms, j = R.ceil(COLS, 64), np.arange(COLS // 16)[None]
    scales = o.scales.cpu().numpy()
    for lo in range(0, ROWS, 250):
        s = slice(lo, lo + 250)
        part, p = N.run(h, fmt, f[s], r[s], pw, nw, None if gt is None else gt[s], gate_ld=COLS if gate else 0)
        assert torch.equal(out[s], part) and torch.equal(o.codes[s], p.codes)
        a = scales[R.scale_at(np.arange(lo, lo + 250)[:, None], j, atoms)]
        b = p.scales.cpu().numpy()[R.scale_at(np.arange(250)[:, None], j, atoms)]
        assert np.array_equal(a, b)


@pytest.mark.parametrize("which", ["r", "f"])
@pytest.mark.parametrize("dt", [synth.F16, synth.BF16])
def test_norm_in_place_over_many_rows(h, dt, which):
    f, r = many(N.TD[dt], 1), many(N.TD[dt], 2)
    w = N.data(1, COLS, N.TD[dt], 3)[0]
    want, o = N.run(h, qg.GEMM_MXFP4, f, r, post=w, pre=w)
    f2, r2 = f.clone(), r.clone()
    got, o2 = N.run(h, qg.GEMM_MXFP4, f2, r2, post=w, pre=w, out=r2 if which == "r" else f2)
    assert torch.equal(got, want) and torch.equal(o.codes, o2.codes) and torch.equal(o.scales, o2.scales)
    assert torch.equal(f2 if which == "r" else r2, f if which == "r" else r)


@pytest.mark.parametrize("fmt", N.FORMATS)
def test_norm_by_expert_over_many_rows(h, fmt):
    # rows 0 .. 199 and 1100 .. belong to nobody: they get their residual alone
    f, r = many(torch.bfloat16, 1), many(torch.bfloat16, 2)
    w = N.data(1, COLS, torch.bfloat16, 3)[0]
    want, o = N.run(h, fmt, f, r, post=w, pre=w)
    off = np.array([200, 700, 700, 701, 1100])
    e = qg.MxOperand(fmt, ROWS, COLS, num_experts=4)
    e.codes.fill_(0xAA)
    offd = torch.from_numpy(off.astype(np.int32)).cuda()
    n = qg.gemm_mx_norm_t(format=fmt, tensor_scale=1.0, eps=1e-5, residual_scale=0.7, pre_weight=qg.ptr(w), post_weight=qg.ptr(w),
                          weight_type=qg.GEMM_BF16, expert_offsets=qg.ptr(offd), num_experts=4)
    out = torch.full_like(want, float("nan"))
    lay = qg.row_major(r)
    assert qg.gemm_mx_norm_quantize(h, n, qg.ptr(f), lay, qg.ptr(r), lay, qg.ptr(out), lay, *e.args(), qg.current_stream()) == 0
    assert torch.equal(out, want) and torch.equal(e.codes[200:1100], o.codes[200:1100])
    assert bool((e.codes[:200] == 0xAA).all()) and bool((e.codes[1100:] == 0xAA).all())
    nb = R.ceil(COLS, R.BLOCK[fmt])
    atoms, j = R.ceil(nb, 4), np.arange(nb)[None]
    a = e.scales.cpu().numpy()[R.scale_at(R.expert_rows(off)[:, None], j, atoms)]
    b = o.scales.cpu().numpy()[R.scale_at(np.arange(200, 1100)[:, None], j, atoms)]
    assert np.array_equal(a, b)


@pytest.mark.parametrize("which", ["r", "f"])
@pytest.mark.parametrize("dt", [synth.F32, synth.F16, synth.BF16])
@pytest.mark.parametrize("off", [0, 1, 3, 6])
@pytest.mark.parametrize("rows,cols", [(9, 1091), (9, 5003), (1100, 2049)])
def test_norm_in_place_on_rows_that_start_anywhere(h, rows, cols, off, dt, which):
    ld, td = cols + 10, N.TD[dt]

    def odd(seed):
        buf = torch.full((rows * ld + 8,), 7.0, dtype=td, device="cuda")
        buf[off:off + rows * ld].view(rows, ld)[:, :cols] = N.data(rows, cols, td, seed)
        return buf, buf[off:off + rows * ld].view(rows, ld)[:, :cols]

    (_, f), (_, r) = odd(1), odd(2)
    w = N.data(1, cols, td, 3)[0]
    want, o = N.run(h, qg.GEMM_NVFP4, f, r, post=w, pre=w)
    (fb, f2), (rb, r2) = odd(1), odd(2)
    got, o2 = N.run(h, qg.GEMM_NVFP4, f2, r2, post=w, pre=w, out=r2 if which == "r" else f2)
    assert torch.equal(got, want) and torch.equal(o.codes, o2.codes) and torch.equal(o.scales, o2.scales)
    for buf in (fb, rb):
        around = buf.clone()
        around[off:off + rows * ld].view(rows, ld)[:, :cols] = 7.0
        assert bool((around == 7).all())
