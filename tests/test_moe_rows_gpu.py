"""Quantisation of rows to int8, placing rows by expert, and the weighted sum
back to tokens, against their definitions."""
import numpy as np
import pytest
import torch

import moe_ref as ref
import quantized_gemm_tcgen05_gb300 as qg

pytestmark = pytest.mark.gpu
INV, UNS, OK = qg.GEMM_ERR_INVALID_ARG, qg.GEMM_ERR_UNSUPPORTED, qg.GEMM_OK


@pytest.fixture(scope="module")
def h():
    h = qg.gemm_create()
    yield h
    qg.gemm_destroy(h)


def values(seed, rows, cols, x="bf16", pad=0, shift=0):
    """[rows, cols] of type x, row stride cols + pad, `shift` elements off alignment."""
    g = torch.Generator().manual_seed(seed)
    flat = torch.randn(rows * (cols + pad) + shift + 64, generator=g).to(ref.TORCH[x]).cuda()
    return flat[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


def quantize(h, x, codes, scales):
    rc = qg.gemm_s8_quantize(h, qg.ptr(x), qg.row_major(x), qg.ptr(codes), qg.row_major(codes), qg.ptr(scales), qg.current_stream())
    assert rc == OK, qg.gemm_status_string(rc)


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,pad,shift,ypad", [
    (1, 1, 0, 0, 0), (3, 16, 0, 0, 0), (5, 17, 0, 0, 15), (4, 515, 2, 1, 0), (7, 4096, 0, 0, 0), (3, 4099, 5, 3, 1), (9, 4112, 16, 0, 0),
    (2, 14336, 8, 4, 16), (2, 32768, 0, 0, 0), (2, 32769, 0, 0, 3), (1, 70001, 3, 2, 0)])
def test_quantize(h, rows, cols, pad, shift, ypad, x):
    v = values(rows + cols, rows, cols, x, pad, shift)
    buf = torch.full((rows * (cols + ypad) + 64,), 77, dtype=torch.int8, device="cuda")
    codes = buf[16:16 + rows * (cols + ypad)].view(rows, cols + ypad)[:, :cols]
    scales = torch.full((rows + 8,), 7.0, device="cuda")
    quantize(h, v, codes, scales)
    q, s = ref.quantize(v)
    assert np.array_equal(codes.cpu().numpy(), q) and np.array_equal(scales[:rows].cpu().numpy(), s)
    # nothing else was written
    rest = buf.clone()
    rest[16:16 + rows * (cols + ypad)].view(rows, cols + ypad)[:, :cols] = 77
    assert (rest == 77).all() and (scales[rows:] == 7).all()


def test_quantize_special_rows(h):
    v = values(1, 12, 100, "f32")
    v[0] = 0.0
    v[1, 3] = torch.nan
    v[2, 99] = torch.inf
    v[3, 0] = -torch.inf
    v[4] *= 2.0 ** -149 / v[4].abs().max() * 3
    v[5] *= 1.5e-36 / v[5].abs().max()
    v[6] *= 1.4e-36 / v[6].abs().max()
    v[7] *= 3.4e38 / v[7].abs().max()
    v[8] = torch.arange(100) - 50.5  # ties
    v[8, 0] = 127.0
    v[9] = -v[8]
    v[10] = -0.0
    codes, scales = torch.empty(12, 100, dtype=torch.int8, device="cuda"), torch.empty(12, device="cuda")
    quantize(h, v, codes, scales)
    q, s = ref.quantize(v)
    assert np.array_equal(codes.cpu().numpy(), q) and np.array_equal(scales.cpu().numpy(), s, equal_nan=True)
    assert (codes[1:4] == 0).all() and scales[1:4].isnan().all()


def test_quantize_matrices(h):
    """Weights of several experts in one call, matrices and rows with gaps."""
    flat = values(3, 3 * 10, 80, "bf16").reshape(3, 10, 80)[:, :7, :65]
    codes = torch.full((3, 9, 96), 77, dtype=torch.int8, device="cuda")
    scales = torch.empty(3, 7, device="cuda")
    quantize(h, flat, codes[:, :7, :65], scales)
    for e in range(3):
        q, s = ref.quantize(flat[e])
        assert np.array_equal(codes[e, :7, :65].cpu().numpy(), q) and np.array_equal(scales[e].cpu().numpy(), s)
    assert (codes[:, 7:] == 77).all() and (codes[:, :, 65:] == 77).all()


def place(seed, tokens, topk, rows, missing=0.0):
    """A map with no row named twice; some entries name none."""
    g = torch.Generator().manual_seed(seed)
    m = torch.randperm(rows, generator=g)[:tokens * topk].int()
    drop = torch.rand(tokens * topk, generator=g) < missing
    bad = torch.tensor([-1, -7, rows, rows + 5, 2 ** 31 - 1], dtype=torch.int32)
    m[drop] = bad[torch.arange(int(drop.sum())) % 5]
    return m.view(tokens, topk).cuda()


@pytest.mark.parametrize("x,to", [("f32", "s8"), ("f16", "s8"), ("bf16", "s8"), ("f32", "f32"), ("bf16", "bf16"), ("s8", "s8"), ("e4m3", "e4m3")])
@pytest.mark.parametrize("tokens,cols,topk,extra", [(1, 64, 1, 0), (16, 4096, 2, 0), (5, 33, 6, 9), (40, 1000, 8, 3), (1030, 72, 3, 5), (3, 20011, 2, 0)])
def test_dispatch(h, tokens, cols, topk, extra, x, to):
    kind = {"s8": torch.int8, "e4m3": torch.float8_e4m3fn, **ref.TORCH}
    v = values(tokens, tokens, cols, "f32", pad=extra)
    if x == "s8":
        v = (v * 30).to(torch.int8)
    else:
        v = v.to(kind[x])
    if x == "bf16" and to == "bf16":
        v[0, 0] = torch.nan
    rows = tokens * topk + extra
    m = place(tokens, tokens, topk, rows, 0.1 if extra else 0.0)
    y = torch.full((rows + 1, cols + extra), 55, dtype=torch.uint8, device="cuda") if to in ("s8", "e4m3") else \
        torch.full((rows + 1, cols + extra), 55.0, dtype=kind[to], device="cuda")
    y = y.view(kind[to])
    s = torch.full((rows + 1,), 55.0, device="cuda")
    quantised = x != to
    out = y[:rows, :cols]
    rc = qg.gemm_moe_dispatch(h, qg.ptr(v), qg.row_major(v), qg.ptr(m), topk, qg.ptr(y), qg.row_major(out), qg.ptr(s) if quantised else None,
                              qg.current_stream())
    assert rc == OK, qg.gemm_status_string(rc)
    want = torch.full_like(y.view(torch.uint8) if y.element_size() == 1 else y.view({2: torch.int16, 4: torch.int32}[y.element_size()]), 0)
    want = want.cpu()
    want[:] = (y[-1:, :1].view(want.dtype)).cpu()
    ws = torch.full((rows + 1,), 55.0)
    if quantised:
        q, sc = ref.quantize(v)
        bits = torch.from_numpy(q).view(torch.uint8)
    else:
        bits = v.cpu().contiguous().view(want.dtype)
    for t in range(tokens):
        for j in range(topk):
            r = int(m[t, j])
            if 0 <= r < rows:
                want[r, :cols] = bits[t]
                if quantised:
                    ws[r] = float(sc[t])
    assert torch.equal(y.view(want.dtype).cpu(), want)
    assert torch.equal(s.cpu(), ws)


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("beta", [0.0, 1.0, -0.5])
@pytest.mark.parametrize("tokens,cols,topk,extra,shift", [(1, 1, 1, 0, 0), (16, 4096, 2, 0, 0), (7, 1033, 5, 3, 1), (33, 264, 8, 0, 0), (130, 40, 32, 6, 0),
                                                          (3, 9000, 4, 0, 4)])
def test_combine(h, tokens, cols, topk, extra, shift, beta, x):
    d = ref.TORCH[x]
    rows = tokens * topk + extra
    y = values(1, rows, cols, x, extra, shift)
    m = place(2, tokens, topk, rows, 0.1 if extra else 0.0)
    w = torch.rand(tokens, topk, generator=torch.Generator().manual_seed(3)).cuda()
    c = values(4, tokens, cols, x, extra, shift)
    out = torch.full((tokens + 1, cols + extra), 5.0, dtype=d, device="cuda")
    rc = qg.gemm_moe_combine(h, qg.ptr(y), qg.row_major(y), qg.ptr(m), qg.ptr(w), topk, beta, qg.ptr(c) if beta else None,
                             qg.row_major(c) if beta else None, qg.ptr(out), qg.row_major(out[:tokens, :cols]), qg.current_stream())
    assert rc == OK, qg.gemm_status_string(rc)
    have = ((m >= 0) & (m < rows)).double().cpu().unsqueeze(-1)
    terms = w.double().cpu().unsqueeze(-1) * y.double().cpu()[m.long().clamp(0, rows - 1).cpu()] * have
    want, size = terms.sum(1), terms.abs().sum(1)
    if beta:
        want, size = want + beta * c.double().cpu(), size + (beta * c.double().cpu()).abs()
    # topk + 1 fused steps in fp32, then one rounding to d
    tol = (topk + 1) * 2.0 ** -24 * size * (1 + 2.0 ** -20) + want.abs() * ref.EPS[d] / 2 * (1 + 2.0 ** -10) + 2.0 ** -25
    if x == "f32":
        tol = (topk + 1) * 2.0 ** -24 * size * (1 + 2.0 ** -20) + 2.0 ** -140
    assert ((out[:tokens, :cols].double().cpu() - want).abs() <= tol).all()
    assert (out[tokens:] == 5).all() and (out[:, cols:] == 5).all()
    if beta:  # in place
        rc = qg.gemm_moe_combine(h, qg.ptr(y), qg.row_major(y), qg.ptr(m), qg.ptr(w), topk, beta, qg.ptr(c), qg.row_major(c), qg.ptr(c),
                                 qg.row_major(c), qg.current_stream())
        assert rc == OK
        assert torch.equal(c, out[:tokens, :cols])


def test_combine_nan_weight_shows_and_nan_c_does_not(h):
    y = values(1, 8, 64, "bf16")
    m = torch.tensor([[0, 1], [-1, -1], [-1, -1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.5], [0.0, 0.0], [torch.nan, torch.nan]], device="cuda")
    c = torch.full((3, 64), torch.nan, dtype=torch.bfloat16, device="cuda")
    out = torch.full((3, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    assert qg.gemm_moe_combine(h, qg.ptr(y), qg.row_major(y), qg.ptr(m), qg.ptr(w), 2, 0.0, qg.ptr(c), qg.row_major(c), qg.ptr(out),
                               qg.row_major(out), qg.current_stream()) == OK
    assert not out[0].isnan().any() and (out[1] == 0).all() and out[2].isnan().all()


def test_empty(h):
    e = torch.empty(0, 64, device="cuda")
    q = torch.empty(0, 64, dtype=torch.int8, device="cuda")
    st = qg.current_stream()
    assert qg.gemm_s8_quantize(h, None, qg.row_major(e), None, qg.row_major(q), None, st) == OK
    assert qg.gemm_moe_dispatch(h, None, qg.row_major(e), None, 2, None, qg.row_major(q), None, st) == OK
    assert qg.gemm_moe_combine(h, None, qg.row_major(e), None, None, 2, 0.0, None, None, None, qg.row_major(e), st) == OK
    # tokens, but no rows anywhere: zeros
    m, w = torch.full((3, 2), -1, dtype=torch.int32, device="cuda"), torch.zeros(3, 2, device="cuda")
    out = torch.full((3, 64), 5.0, device="cuda")
    x = torch.ones(3, 64, device="cuda")
    assert qg.gemm_moe_dispatch(h, qg.ptr(x), qg.row_major(x), qg.ptr(m), 2, None, qg.row_major(e), None, st) == OK
    assert qg.gemm_moe_combine(h, None, qg.row_major(e), qg.ptr(m), qg.ptr(w), 2, 0.0, None, None, qg.ptr(out), qg.row_major(out), st) == OK
    assert (out == 0).all()


def test_refusals(h):
    x = torch.ones(8, 64, device="cuda")
    q, s = torch.full((16, 64), 9, dtype=torch.int8, device="cuda"), torch.full((16,), 9.0, device="cuda")
    y, c = torch.full((16, 64), 9.0, device="cuda"), torch.ones(8, 64, device="cuda")
    m, w = torch.arange(16, dtype=torch.int32, device="cuda"), torch.ones(16, device="cuda")
    host = torch.zeros(4096)
    hp = host.data_ptr()
    st = qg.current_stream()
    lay = lambda t, **kw: qg.gemm_layout_t(**{**{f: getattr(qg.row_major(t), f) for f, _ in qg.gemm_layout_t._fields_}, **kw})  # noqa: E731
    quant = dict(X=qg.ptr(x), Xdesc=qg.row_major(x), Q=qg.ptr(q), Qdesc=lay(q, rows=8), S=qg.ptr(s))
    disp = dict(X=qg.ptr(x), Xdesc=qg.row_major(x), rows=qg.ptr(m), topk=2, Y=qg.ptr(q), Ydesc=qg.row_major(q), S=qg.ptr(s))
    comb = dict(Y=qg.ptr(y), Ydesc=qg.row_major(y), rows=qg.ptr(m), weights=qg.ptr(w), topk=2, beta=1.0, C=qg.ptr(c), Cdesc=qg.row_major(c),
                D=qg.ptr(x), Ddesc=qg.row_major(x))
    common_q = [(dict(X=None), INV), (dict(X=hp), INV), (dict(X=quant["X"] + 2), INV), (dict(Xdesc=None), INV), (dict(S=None), INV), (dict(S=hp), INV),
                (dict(S=quant["S"] + 2), INV), (dict(Xdesc=lay(x, order=1)), UNS), (dict(Xdesc=lay(x, type=qg.GEMM_S4)), UNS),
                (dict(Xdesc=lay(x, ld=63)), INV), (dict(Xdesc=lay(x, cols=63)), INV), (dict(Xdesc=lay(x, rows=-1)), INV)]
    for change, want in common_q + [(dict(Q=None), INV), (dict(Q=hp), INV), (dict(Qdesc=None), INV), (dict(Qdesc=lay(q)), INV),
                                    (dict(Qdesc=lay(q, rows=8, type=qg.GEMM_F32)), UNS), (dict(Xdesc=lay(x, type=qg.GEMM_S8)), UNS),
                                    (dict(Qdesc=lay(q, rows=8, num=2, batch_stride=512)), INV),
                                    (dict(Xdesc=lay(x, num=2, batch_stride=1), Qdesc=lay(q, rows=8, num=2, batch_stride=512)), INV)]:
        rc = qg.gemm_s8_quantize(h, *({**quant, **change}).values(), st)
        assert rc == want, ("quantize", change, rc)
    for change, want in common_q + [(dict(rows=None), INV), (dict(rows=hp), INV), (dict(rows=disp["rows"] + 1), INV), (dict(topk=0), INV),
                                    (dict(topk=33), INV), (dict(Y=None), INV), (dict(Ydesc=None), INV), (dict(Ydesc=lay(q, type=qg.GEMM_F16)), UNS),
                                    (dict(Ydesc=lay(q, num=2, batch_stride=1024)), UNS)]:
        rc = qg.gemm_moe_dispatch(h, *({**disp, **change}).values(), st)
        assert rc == want, ("dispatch", change, rc)
    for change, want in [(dict(Y=None), INV), (dict(Y=hp), INV), (dict(Ydesc=None), INV), (dict(rows=None), INV), (dict(weights=None), INV),
                         (dict(weights=hp), INV), (dict(topk=0), INV), (dict(topk=33), INV), (dict(C=None), INV), (dict(Cdesc=None), INV),
                         (dict(D=None), INV), (dict(Ddesc=None), INV), (dict(D=comb["D"] + 2), INV), (dict(Cdesc=lay(c, rows=7)), INV),
                         (dict(Cdesc=lay(c, type=qg.GEMM_F16)), UNS), (dict(Ydesc=lay(y, cols=32)), INV), (dict(Ydesc=lay(y, type=qg.GEMM_BF16)), UNS),
                         (dict(Ddesc=lay(x, type=qg.GEMM_S8), Ydesc=lay(y, type=qg.GEMM_S8)), UNS), (dict(Ydesc=lay(y, num=2, batch_stride=512)), UNS)]:
        rc = qg.gemm_moe_combine(h, *({**comb, **change}).values(), st)
        assert rc == want, ("combine", change, rc)
    torch.cuda.synchronize()
    assert (q == 9).all() and (s == 9).all() and (x == 1).all() and (y == 9).all()
