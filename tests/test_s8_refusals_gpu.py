"""What the int8 products refuse: a status returned by the host before anything
is enqueued; D keeps what it held."""
import pytest
import torch

import quantized_gemm_tcgen05_gb300 as qg

pytestmark = pytest.mark.gpu
INV, UNS, OK = qg.GEMM_ERR_INVALID_ARG, qg.GEMM_ERR_UNSUPPORTED, qg.GEMM_OK


@pytest.fixture(scope="module")
def h():
    h = qg.gemm_create()
    yield h
    qg.gemm_destroy(h)


def ld(d, **kw):
    return qg.gemm_layout_t(**{**{f: getattr(d, f) for f, _ in d._fields_}, **kw})


@pytest.mark.parametrize("experts", [0, 2])
def test_refusals(h, experts):
    m, n, k = 32, 64, 128
    a = torch.zeros(m, k, dtype=torch.int8, device="cuda")
    b = torch.zeros(*((experts,) if experts else ()), n, k, dtype=torch.int8, device="cuda")
    sa, sb = torch.ones(m, device="cuda"), torch.ones(2 * n, device="cuda")
    d, c = torch.full((m, n), 4.0, dtype=torch.bfloat16, device="cuda"), torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    bias = torch.zeros(n, device="cuda")
    off = torch.tensor([0, 10, 32], dtype=torch.int32, device="cuda")
    hp = torch.zeros(1 << 16, dtype=torch.uint8).data_ptr()
    good = dict(op=qg.gemm_op_t(), alpha=1.0, A=qg.ptr(a), Adesc=qg.row_major(a), SA=qg.ptr(sa), B=qg.ptr(b), Bdesc=qg.col_major_from_nk(b),
                SB=qg.ptr(sb), beta=0.0, C=None, Cdesc=None, D=qg.ptr(d), Ddesc=qg.row_major(d))
    if experts:
        good.update(off=qg.ptr(off), experts=experts)
    call = qg.gemm_run_s8_grouped if experts else qg.gemm_run_s8
    assert call(h, *good.values(), qg.current_stream()) == OK
    torch.cuda.synchronize()
    d.fill_(4.0)
    op = lambda **kw: dict(op=qg.gemm_op_t(**kw))  # noqa: E731
    A, B, D = good["Adesc"], good["Bdesc"], good["Ddesc"]
    with_c = dict(beta=1.0, C=qg.ptr(c), Cdesc=qg.row_major(c))
    cases = [
        (dict(op=None), INV), (dict(A=None), INV), (dict(B=None), INV), (dict(D=None), INV), (dict(A=hp), INV), (dict(B=hp), INV), (dict(D=hp), INV),
        (dict(SA=hp), INV), (dict(SB=hp), INV), (dict(SA=good["SA"] + 2), INV), (dict(A=good["A"] + 8), INV), (dict(B=good["B"] + 4), INV),
        (dict(D=good["D"] + 1), INV), (dict(Adesc=None), INV), (dict(Bdesc=None), INV), (dict(Ddesc=None), INV),
        (dict(Adesc=ld(A, type=qg.GEMM_E4M3)), UNS), (dict(Bdesc=ld(B, type=qg.GEMM_S4)), UNS), (dict(Adesc=ld(A, order=1)), UNS),
        (dict(Bdesc=ld(B, order=0)), UNS), (dict(Ddesc=ld(D, type=qg.GEMM_S8)), UNS), (dict(Ddesc=ld(D, order=1)), UNS),
        (dict(Adesc=ld(A, ld=127)), INV), (dict(Adesc=ld(A, ld=136)), INV), (dict(Bdesc=ld(B, ld=132)), INV), (dict(Ddesc=ld(D, ld=63)), INV),
        (dict(Ddesc=ld(D, rows=31)), INV), (dict(Ddesc=ld(D, cols=63)), INV), (dict(Bdesc=ld(B, rows=127)), INV),
        (dict(Adesc=ld(A, cols=131072, ld=131072), Bdesc=ld(B, rows=131072, ld=131072, batch_stride=131072 * n)), UNS),
        (dict(beta=1.0), INV), (dict(with_c, Cdesc=None), INV), (dict(with_c, C=hp), INV), (dict(with_c, Cdesc=ld(D, type=qg.GEMM_F16)), UNS),
        (dict(with_c, Cdesc=ld(D, ld=63)), INV), (dict(with_c, Cdesc=ld(D, num=2, batch_stride=m * n)), INV),
        (op(epilogue=8), INV), (op(epilogue=6), INV), (op(epilogue=1), INV), (op(epilogue=1, bias=qg.ptr(bias), bias_type=qg.GEMM_S8), UNS),
        (op(epilogue=1, bias=hp), INV), (op(epilogue=1, bias=qg.ptr(bias) + 2), INV), (op(dispatch=3), INV), (op(splitk=-1), INV), (op(splitk=3), UNS),
        (op(splitk=16), UNS), (op(streamk=2), INV), (op(streamk=1), UNS), (op(splitk=2, streamk=1), INV), (op(quant_a_group=64), UNS),
        (op(quant_b_group=64), UNS), (op(b_zero=qg.ptr(bias)), UNS),
        (dict(Adesc=ld(A, num=2, batch_stride=m * k)), INV if experts else UNS),
        (dict(Bdesc=ld(B, num=3, batch_stride=n * k)), INV if experts else UNS),
    ]
    if experts:
        cases += [(dict(off=None), INV), (dict(off=hp), INV), (dict(off=good["off"] + 2), INV), (dict(experts=0), INV), (dict(experts=4097), INV),
                  (dict(experts=3), INV), (dict(Bdesc=ld(B, batch_stride=n * k - 16)), INV), (dict(Bdesc=ld(B, batch_stride=n * k + 8)), INV)]
    for change, want in cases:
        rc = call(h, *{**good, **change}.values(), qg.current_stream())
        assert rc == want, (change, rc)
    torch.cuda.synchronize()
    assert (d == 4).all()
