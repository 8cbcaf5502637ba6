"""What the 4-bit microscaled calls refuse: every refusal is a status returned
by the host before anything is enqueued, and the outputs keep what they held."""
import pytest
import torch

import quantized_gemm_tcgen05_gb300 as qg

pytestmark = pytest.mark.gpu

INV, UNS, OK = qg.GEMM_ERR_INVALID_ARG, qg.GEMM_ERR_UNSUPPORTED, qg.GEMM_OK
NV = qg.GEMM_NVFP4


@pytest.fixture(scope="module")
def h():
    h = qg.gemm_create()
    yield h
    qg.gemm_destroy(h)


class Case:
    """A call that is accepted as it stands; tests change one thing."""

    def __init__(self):
        self.m, self.n, self.k = 32, 64, 128
        self.A, self.B = qg.MxOperand(NV, self.m, self.k), qg.MxOperand(NV, self.n, self.k)
        self.D = torch.full((self.m, self.n), 4.0, dtype=torch.bfloat16, device="cuda")
        self.C = torch.zeros_like(self.D)
        self.bias = torch.zeros(self.n, device="cuda")
        self.off = torch.tensor([0, 10, 32], dtype=torch.int32, device="cuda")

    def product(self):
        a, al, sa, sas = self.A.args()
        b, bl, sb, sbs = self.B.args(b=True)
        return dict(op=qg.gemm_op_t(), format=NV, alpha=1.0, A=a, Adesc=al, SA=sa, SA_size=sas, B=b, Bdesc=bl, SB=sb,
                    SB_size=sbs, beta=0.0, C=None, Cdesc=None, D=qg.ptr(self.D), Ddesc=qg.row_major(self.D),
                    stream=qg.current_stream())


def ld(d, **kw):
    vals = {f: getattr(d, f) for f, _ in d._fields_}
    vals.update(kw)
    return qg.gemm_layout_t(**vals)


def test_product_refusals(h):
    c = Case()
    good = c.product()
    assert qg.gemm_run_mx(h, **good) == OK
    torch.cuda.synchronize()
    c.D.fill_(4.0)
    host = torch.zeros(1 << 16, dtype=torch.uint8)
    op = lambda **kw: dict(op=qg.gemm_op_t(**kw))  # noqa: E731
    Ad, Bd, Dd = good["Adesc"], good["Bdesc"], good["Ddesc"]
    cases = [
        (dict(format=0), UNS), (dict(format=3), UNS),
        (dict(A=None), INV), (dict(B=None), INV), (dict(SA=None), INV), (dict(SB=None), INV), (dict(D=None), INV),
        (dict(Adesc=None), INV), (dict(Bdesc=None), INV), (dict(Ddesc=None), INV),
        (dict(A=good["A"] + 8), INV), (dict(SB=good["SB"] + 4), INV), (dict(D=good["D"] + 1), INV),
        (dict(A=host.data_ptr()), INV), (dict(D=host.data_ptr()), INV), (dict(SA=host.data_ptr()), INV),
        (dict(SA_size=good["SA_size"] - 1), INV), (dict(SB_size=0), INV),
        (dict(Adesc=ld(Ad, ld=144)), INV), (dict(Adesc=ld(Ad, ld=96)), INV), (dict(Adesc=ld(Ad, type=qg.GEMM_E4M3)), UNS),
        (dict(Adesc=ld(Ad, order=1)), UNS), (dict(Adesc=ld(Ad, rows=-1)), INV), (dict(Adesc=ld(Ad, rows=33)), INV),
        (dict(Adesc=ld(Ad, num=2, batch_stride=1 << 14)), UNS), (dict(Bdesc=ld(Bd, num=2, batch_stride=1 << 14)), INV),
        (dict(Bdesc=ld(Bd, rows=64)), INV), (dict(Bdesc=ld(Bd, order=0)), UNS),
        (dict(Ddesc=ld(Dd, type=qg.GEMM_S8)), UNS), (dict(Ddesc=ld(Dd, ld=63)), INV), (dict(Ddesc=ld(Dd, cols=63)), INV),
        (dict(beta=1.0), INV), (dict(beta=1.0, C=qg.ptr(c.C), Cdesc=ld(Dd, type=qg.GEMM_F32)), UNS),
        (dict(beta=1.0, C=host.data_ptr(), Cdesc=Dd), INV),
        (op(epilogue=8), INV), (op(epilogue=6), INV), (op(epilogue=1), INV),
        (op(epilogue=1, bias=qg.ptr(c.bias), bias_type=qg.GEMM_S8), UNS),
        (op(epilogue=1, bias=qg.ptr(c.bias) + 2, bias_type=qg.GEMM_F32), INV),
        (op(splitk=3), UNS), (op(splitk=16), UNS), (op(splitk=-1), INV), (op(streamk=1), UNS), (op(streamk=2), INV),
        (op(quant_a_group=64), UNS), (op(quant_b_group=64), UNS), (op(b_zero=qg.ptr(c.bias)), UNS), (op(dispatch=3), INV),
    ]
    for change, want in cases:
        assert qg.gemm_run_mx(h, **{**good, **change}) == want, change
    assert qg.gemm_run_mx(None, **good) == INV
    torch.cuda.synchronize()
    assert bool((c.D == 4).all())
    # nothing to do is no error
    empty = dict(Adesc=ld(Ad, rows=0), Ddesc=ld(Dd, rows=0))
    assert qg.gemm_run_mx(h, **{**good, **empty}) == OK and qg.gemm_last_choice(h) == "empty"


def test_grouped_refusals(h):
    c = Case()
    w = qg.MxOperand(NV, c.n, c.k, num=2)
    a = qg.MxOperand(NV, c.m, c.k, num_experts=2)
    good = c.product()
    good["A"], good["Adesc"], good["SA"], good["SA_size"] = a.args()
    good["B"], good["Bdesc"], good["SB"], good["SB_size"] = w.args(b=True)
    good.update(expert_alpha=None, expert_offsets_dev=qg.ptr(c.off), num_experts=2)
    assert qg.gemm_run_mx_grouped(h, **good) == OK
    torch.cuda.synchronize()
    c.D.fill_(4.0)
    for change, want in [
        (dict(expert_offsets_dev=None), INV), (dict(num_experts=0), INV), (dict(num_experts=3), INV),
        (dict(num_experts=5000), INV), (dict(expert_offsets_dev=qg.ptr(c.off) + 1), INV),
        (dict(expert_alpha=qg.ptr(c.bias) + 2), INV), (dict(SA_size=good["SA_size"] - 1), INV),
        (dict(SB_size=good["SB_size"] - 1), INV), (dict(Bdesc=ld(good["Bdesc"], batch_stride=128)), INV),
        (dict(Bdesc=ld(good["Bdesc"], batch_stride=64 * 128 + 16)), INV),
        (dict(expert_offsets_dev=torch.zeros(3, dtype=torch.int32).data_ptr()), INV),
    ]:
        assert qg.gemm_run_mx_grouped(h, **{**good, **change}) == want, change
    torch.cuda.synchronize()
    assert bool((c.D == 4).all())


def test_quantize_refusals(h):
    x = torch.ones(32, 128, dtype=torch.bfloat16, device="cuda")
    o = qg.MxOperand(NV, 32, 128)
    q, ql, s, sb = o.args()
    xl = qg.row_major(x)
    off = torch.tensor([0, 32], dtype=torch.int32, device="cuda")
    good = dict(format=NV, tensor_scale=1.0, X=qg.ptr(x), Xdesc=xl, Q=q, Qdesc=ql, S=s, S_size=sb,
                expert_offsets_dev=None, num_experts=0, stream=qg.current_stream())
    out = torch.empty(32, 128, dtype=torch.float32, device="cuda")
    back = dict(format=NV, tensor_scale=1.0, Q=q, Qdesc=ql, S=s, S_size=sb, D=qg.ptr(out), Ddesc=qg.row_major(out),
                expert_offsets_dev=None, num_experts=0, stream=qg.current_stream())
    assert qg.gemm_mx_quantize(h, **good) == OK and qg.gemm_mx_dequantize(h, **back) == OK
    o.codes.fill_(1)
    for change, want in [
        (dict(format=0), UNS), (dict(tensor_scale=0.0), INV), (dict(tensor_scale=-1.0), INV),
        (dict(tensor_scale=float("nan")), INV), (dict(tensor_scale=float("inf")), INV),
        (dict(format=qg.GEMM_MXFP4, tensor_scale=2.0), INV), (dict(Qdesc=ld(ql, ld=144)), INV),
        (dict(Qdesc=ld(ql, type=qg.GEMM_S4)), UNS), (dict(Qdesc=ld(ql, cols=127)), INV), (dict(Q=q + 8), INV),
        (dict(S=s + 8), INV), (dict(S_size=sb - 1), INV), (dict(expert_offsets_dev=qg.ptr(off)), INV),
        (dict(num_experts=1), INV), (dict(S=None), INV), (dict(Q=None), INV), (dict(Qdesc=None), INV),
    ]:
        assert qg.gemm_mx_quantize(h, **{**good, **change}) == want, change
        assert qg.gemm_mx_dequantize(h, **{**back, **change}) == want, change
    for change, want in [(dict(Xdesc=ld(xl, type=qg.GEMM_E4M3)), UNS), (dict(Xdesc=ld(xl, ld=100)), INV),
                         (dict(X=qg.ptr(x) + 1), INV), (dict(Xdesc=None), INV), (dict(X=None), INV),
                         (dict(Xdesc=ld(xl, num=2, batch_stride=0)), INV), (dict(Xdesc=ld(xl, order=1)), UNS),
                         (dict(X=torch.zeros(4096).data_ptr()), INV)]:
        assert qg.gemm_mx_quantize(h, **{**good, **change}) == want, change
    assert qg.gemm_mx_dequantize(h, **{**back, "Ddesc": ld(qg.row_major(out), type=qg.GEMM_E5M2)}) == UNS
    torch.cuda.synchronize()
    assert bool((o.codes == 1).all())
    assert qg.gemm_mx_quantize(h, **{**good, "Xdesc": ld(xl, rows=0), "Qdesc": ld(ql, rows=0)}) == OK


def test_norm_refusals(h):
    r = torch.ones(8, 128, dtype=torch.float16, device="cuda")
    f, out, w = r.clone(), torch.full_like(r, 4.0), torch.ones(128, dtype=torch.float16, device="cuda")
    o = qg.MxOperand(NV, 8, 128)
    q, ql, s, sb = o.args()
    rl = qg.row_major(r)
    base = dict(format=NV, tensor_scale=1.0, eps=1e-5, residual_scale=1.0, weight_type=qg.GEMM_F16,
                pre_weight=qg.ptr(w), post_weight=qg.ptr(w), gate=qg.ptr(w), gate_type=qg.GEMM_F16, gate_ld=0)
    n = lambda **kw: qg.gemm_mx_norm_t(**{**base, **kw})  # noqa: E731
    good = dict(op=n(), F=qg.ptr(f), Fdesc=rl, R=qg.ptr(r), Rdesc=rl, O=qg.ptr(out), Odesc=rl, Q=q, Qdesc=ql, S=s,
                S_size=sb, stream=qg.current_stream())
    assert qg.gemm_mx_norm_quantize(h, **good) == OK
    torch.cuda.synchronize()
    out.fill_(4.0)
    for change, want in [
        (dict(op=n(format=0)), UNS), (dict(op=n(tensor_scale=0.0)), INV), (dict(op=n(eps=-1.0)), INV),
        (dict(op=n(eps=float("nan"))), INV), (dict(op=n(residual_scale=float("inf"))), INV),
        (dict(op=n(weight_type=qg.GEMM_S8)), UNS), (dict(op=n(gate_type=qg.GEMM_S8)), UNS), (dict(op=n(gate_ld=64)), INV), (dict(op=n(num_experts=1)), INV), (dict(op=n(expert_offsets=qg.ptr(w))), INV),
        (dict(op=n(pre_weight=qg.ptr(w) + 1)), INV), (dict(F=None), INV), (dict(O=None), INV), (dict(R=None), INV),
        (dict(Fdesc=None), INV), (dict(Rdesc=None), INV), (dict(Odesc=ld(rl, type=qg.GEMM_F32, ld=128)), UNS),
        (dict(Fdesc=ld(rl, type=qg.GEMM_BF16)), UNS), (dict(Fdesc=ld(rl, rows=7)), INV), (dict(Qdesc=ld(ql, ld=144)), INV),
        (dict(Rdesc=ld(rl, type=qg.GEMM_E4M3)), UNS), (dict(S_size=sb - 1), INV), (dict(R=qg.ptr(r) + 1), INV),
        (dict(Odesc=ld(rl, num=2, batch_stride=4096)), UNS),
    ]:
        assert qg.gemm_mx_norm_quantize(h, **{**good, **change}) == want, change
    wide = qg.layout(qg.GEMM_F16, 0, 1, 32769, 32784)
    wideq = qg.layout(qg.GEMM_E2M1, 0, 1, 32769, 32800)
    assert qg.gemm_mx_norm_quantize(h, **{**good, "Fdesc": wide, "Rdesc": wide, "Odesc": wide, "Qdesc": wideq}) == UNS
    torch.cuda.synchronize()
    assert bool((out == 4).all())
