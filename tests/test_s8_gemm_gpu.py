"""Int8 products: sums are exact and the fp32 steps after them are stated, so
every result but GELU's is compared bit for bit, on every kernel."""
import math
import os

import numpy as np
import pytest
import torch

import moe_ref as ref
import quantized_gemm_tcgen05_gb300 as qg

pytestmark = pytest.mark.gpu
OK = qg.GEMM_OK
KERNELS = ["", "s8_gemv", "s8_t32", "s8_t128", "s8_pair"]


@pytest.fixture(scope="module")
def h():
    h = qg.gemm_create()
    yield h
    assert qg.gemm_device_status(h, qg.current_stream()) == OK
    qg.gemm_destroy(h)


@pytest.fixture
def pin():
    def set_(name):
        os.environ["GEMM_FORCE_KERNEL"] = name
    yield set_
    os.environ.pop("GEMM_FORCE_KERNEL", None)


def codes(gen, *shape, ld=None, lo=-128, hi=128):
    """int8 [.., rows, k] in rows of `ld` bytes whose padding is not zero."""
    k = shape[-1]
    ld = -(-k // 16) * 16 if ld is None else ld
    full = torch.randint(-128, 128, (*shape[:-1], ld), generator=gen, dtype=torch.int8)
    full[..., :k] = torch.randint(lo, hi, shape, generator=gen, dtype=torch.int8)
    return full.cuda()[..., :k]


class Problem:
    def __init__(self, m, n, k, d="bf16", seed=0, beta=0.0, act="", bias="f32", scales=True, lda=None, ldb=None, ldd=None, lo=-128, hi=128,
                 sizes=None, alpha=1.5, shift=0):
        g = torch.Generator().manual_seed(seed)
        self.m, self.n, self.k, self.d, self.alpha, self.beta, self.act = m, n, k, ref.TORCH[d], alpha, beta, act
        self.sizes = sizes
        e = len(sizes) if sizes else 0
        self.a = codes(g, m, k, ld=lda, lo=lo, hi=hi)
        self.b = codes(g, *((e,) if e else ()), n, k, ld=ldb, lo=lo, hi=hi)
        self.sa = (torch.rand(m, generator=g) * 0.01 + 1e-3).cuda() if scales else None
        self.sb = (torch.rand(*((e,) if e else ()), n, generator=g) * 0.01 + 1e-3).cuda() if scales else None
        self.bias = torch.randn(n, generator=g).to(ref.TORCH[bias]).cuda() if act else None
        self.ldd = n if ldd is None else ldd
        self.c = torch.randn(m, self.ldd, generator=g).to(self.d).cuda()[:, :n] if beta else None
        self.flat = torch.full((shift + (m + 2) * self.ldd,), 7.0, dtype=self.d, device="cuda")
        self.out = self.flat[shift:].view(m + 2, self.ldd)
        self.off = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda") if e else None

    def run(self, h, splitk=0, stream=None):
        op = qg.gemm_op_t(splitk=splitk)
        if self.act:
            op.epilogue = qg.GEMM_EPILOGUE_BIAS | {"bias": 0, "relu": qg.GEMM_EPILOGUE_RELU, "gelu": qg.GEMM_EPILOGUE_GELU}[self.act]
            op.bias, op.bias_type = qg.ptr(self.bias), qg._dtype_code(self.bias.dtype)
        args = (h, op, self.alpha, qg.ptr(self.a), qg.row_major(self.a), qg.ptr(self.sa), qg.ptr(self.b), qg.col_major_from_nk(self.b),
                qg.ptr(self.sb), self.beta, qg.ptr(self.c), None if self.c is None else qg.row_major(self.c), qg.ptr(self.out),
                qg.row_major(self.out[:self.m, :self.n]))
        st = stream or qg.current_stream()
        rc = qg.gemm_run_s8_grouped(*args, qg.ptr(self.off), len(self.sizes), st) if self.sizes else qg.gemm_run_s8(*args, st)
        assert rc == OK, qg.gemm_status_string(rc)
        return self.out

    def part(self, rows, b, sb):
        act = None if self.act == "gelu" else self.act
        v = ref.product(ref.sums(self.a[rows], b), self.alpha, None if self.sa is None else self.sa[rows], sb,
                        torch.float32 if self.act == "gelu" else self.d, self.beta, None if self.c is None else self.c[rows],
                        self.bias, act == "relu")
        return v

    def expected(self):
        if not self.sizes:
            return self.part(slice(0, self.m), self.b, self.sb)
        out = torch.full((self.m, self.n), 7.0, dtype=torch.float32 if self.act == "gelu" else self.d)
        off = self.off.tolist()
        for e in range(len(self.sizes)):
            if self.sizes[e]:
                mine = slice(off[e], off[e + 1])
                out[mine] = self.part(mine, self.b[e], None if self.sb is None else self.sb[e])
        return out

    def check(self, h, **kw):
        got, want = self.run(h, **kw).cpu(), self.expected()
        y = got[:self.m, :self.n]
        held = self.m if not self.sizes else sum(self.sizes)
        if self.act == "gelu":
            x = want[:held].double()
            e = x * torch.special.ndtr(x)
            if self.d == torch.float32:
                # erff within 2^-22, 1 + erf and the two products rounded
                tol = x.abs() * 2.0 ** -22 * 1.5 + 2.0 ** -140
            else:
                # 2e-5 relative, 0 from -13 on, one rounding (fp16: a subnormal one too)
                tol = e.abs() * (2e-5 + ref.EPS[self.d] / 2 * 1.0001) + 2.0 ** -25 + (x < -13) * x.abs() * 1e-30
            assert ((y[:held].double() - e).abs() <= tol).all()
        else:
            assert torch.equal(y[:held], want[:held])
        assert (y[held:] == 7).all() and (got[self.m:] == 7).all() and (got[:, self.n:] == 7).all()
        assert (self.flat[:self.flat.numel() - self.out.numel()] == 7).all()


SHAPES = [(1, 1, 1), (1, 128, 16), (1, 4096, 2048), (2, 130, 100), (3, 4, 4099), (7, 257, 1000), (8, 1000, 333), (9, 64, 64), (16, 513, 1025),
          (17, 128, 128), (33, 300, 2200), (64, 1030, 520), (65, 96, 1500), (100, 2, 700), (128, 256, 1024), (129, 384, 3000), (200, 1000, 1111),
          (300, 70, 4096), (513, 640, 256)]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("d", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_shapes(h, pin, kernel, m, n, k, d):
    pin(kernel)
    Problem(m, n, k, d, seed=m + n + k).check(h)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("d", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act,beta,bias", [("", 0.5, "f32"), ("bias", 0.0, "f16"), ("relu", 0.0, "bf16"), ("relu", -2.0, "f32"), ("gelu", 0.0, "bf16"),
                                           ("gelu", 1.0, "f32")])
@pytest.mark.parametrize("m,n,k", [(1, 516, 700), (5, 100, 260), (40, 333, 1300), (150, 264, 2080), (260, 512, 300)])
def test_epilogue(h, pin, kernel, m, n, k, act, beta, bias, d):
    pin(kernel)
    Problem(m, n, k, d, seed=m, beta=beta, act=act, bias=bias, alpha=0.01).check(h)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("lo,hi", [(127, 128), (-128, -127)])
@pytest.mark.parametrize("m,n,k", [(2, 40, 70001), (40, 40, 14336), (150, 300, 9000), (300, 520, 5000)])
def test_largest_sums(h, pin, kernel, m, n, k, lo, hi):
    """All codes at an end of the range: sums far beyond what fp32 adds up exactly."""
    pin(kernel)
    p = Problem(m, n, k, "f32", scales=False, lo=lo, hi=hi, alpha=1.0)
    p.a[0, 5] = -3  # a sum that fp32 would lose
    p.a[m - 1] = torch.randint(-128, 128, (k,), dtype=torch.int8, device="cuda")
    p.check(h)


def test_largest_k(h):
    Problem(3, 20, 131071, "f32", scales=False, lo=-128, hi=-127, alpha=1.0).check(h)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("m", [1, 30, 140, 280])
def test_strides_and_nothing_else_written(h, pin, kernel, m):
    pin(kernel)
    for n, ldd, shift in ((200, 203, 1), (256, 272, 0), (77, 77, 3)):
        Problem(m, n, 300, "bf16", lda=512, ldb=320, ldd=ldd, shift=shift, beta=1.0).check(h)
        Problem(m, n, 300, "f32", lda=304, ldb=336, ldd=ldd, shift=shift).check(h)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("sizes,n,k", [([1], 64, 64), ([0, 5, 0, 0, 3], 130, 300), ([16, 0, 40, 1, 9], 257, 1100), ([200, 0, 3, 129, 64], 300, 520),
                                       ([0, 0], 64, 64), ([1] * 40, 96, 160), ([300, 20, 700], 512, 384)])
def test_grouped(h, pin, kernel, sizes, n, k):
    pin(kernel)
    m = sum(sizes)
    for d in ("bf16", "f32"):
        Problem(m + 3, n, k, d, sizes=sizes, seed=m).check(h)  # three rows that no expert holds
    if m:
        Problem(m, n, k, "f16", sizes=sizes, seed=m, beta=0.5, act="gelu", alpha=0.01).check(h)


@pytest.mark.parametrize("kernel", KERNELS)
def test_offsets_that_are_no_partition(h, pin, kernel):
    """Stray offsets lead past neither the operands nor D."""
    pin(kernel)
    for off in ([-5, 3, 2, 1000, 40], [0, 2 ** 30, 2 ** 31 - 1, 0, 40], [60, 50, 40, 30, 20], [40, 40, 40, 40, 40], [-2 ** 31, 2 ** 31 - 1, 0, 0, 0]):
        p = Problem(40, 96, 200, "bf16", sizes=[10, 10, 10, 10])
        p.off.copy_(torch.tensor(off, dtype=torch.int32))
        out = p.run(h)
        torch.cuda.synchronize()
        assert (out[40:] == 7).all() and qg.gemm_device_status(h, qg.current_stream()) == OK


def test_no_k_and_empty(h):
    p = Problem(5, 33, 16, "f32", beta=2.0, act="bias")
    p.a, p.b = p.a[:, :0], p.b[:, :0]
    p.k = 0
    out = p.run(h).cpu()
    want = (2.0 * p.c.cpu() + p.bias.cpu())
    assert torch.equal(out[:5], want)
    e = torch.empty(0, 16, dtype=torch.int8, device="cuda")
    d = torch.empty(0, 8, device="cuda")
    b = torch.zeros(8, 16, dtype=torch.int8, device="cuda")
    assert qg.gemm_run_s8(h, qg.gemm_op_t(), 1.0, None, qg.row_major(e), None, qg.ptr(b), qg.col_major_from_nk(b), None, 0.0, None, None, None,
                          qg.row_major(d), qg.current_stream()) == OK


def test_nan_scales_show(h):
    p = Problem(4, 40, 64, "bf16")
    p.sa[2] = torch.nan
    p.sb[7] = torch.nan
    out = p.run(h)[:4, :40].isnan().cpu()
    want = torch.zeros(4, 40, dtype=torch.bool)
    want[2], want[:, 7] = True, True
    assert torch.equal(out, want)


@pytest.mark.parametrize("splitk", [1, 2, 4, 8])
@pytest.mark.parametrize("m,n,k", [(1, 200, 5000), (20, 128, 2500), (70, 300, 1000), (128, 130, 200), (5, 64, 100)])
def test_k_slices(h, splitk, m, n, k):
    Problem(m, n, k, "f32", beta=1.0).check(h, splitk=splitk)


@pytest.mark.parametrize("m,n,k", [(1, 512, 512), (24, 500, 2000), (300, 512, 1024)])
def test_graph_and_stream(h, m, n, k):
    side = torch.cuda.Stream()
    p = Problem(m, n, k)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        p.run(h)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            p.run(h)
        p.out.fill_(7.0)
        p.a.copy_(codes(torch.Generator().manual_seed(99), m, k))
        for _ in range(3):
            g.replay()
        side.synchronize()
    assert torch.equal(p.out[:m, :n].cpu(), p.expected())


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("m,n,k", [(1, 4096, 14336), (31, 8192, 4096), (130, 2048, 8192)])
def test_cold_operands_back_to_back(h, pin, kernel, m, n, k):
    """Operands that come from far (copies land late and out of order), launches that overlap."""
    pin(kernel)
    ps = [Problem(m, n, k, "f32", seed=i) for i in range(3)]
    flush = torch.empty(160 << 20, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        flush.zero_()
        for p in ps:
            p.run(h)
    for p in ps:
        assert torch.equal(p.out[:m, :n].cpu(), p.expected())


def test_offsets_beyond_32_bits(h):
    """Rows of A, B and D that lie more than 2^32 bytes apart."""
    k, n, m = 64, 40, 3
    ld = (1 << 32) // 2 + 16
    big = torch.zeros(2 * ld + k, dtype=torch.int8, device="cuda")
    p = Problem(m, n, k)
    for i in range(m):
        big[i * ld:i * ld + k] = p.a[i]
    p.a = big.as_strided((m, k), (ld, 1))
    p.check(h)
    rows = torch.zeros(2 * ld + 64, dtype=torch.bfloat16, device="cuda")
    out = rows.as_strided((m, n), (ld, 1))
    op = qg.gemm_op_t()
    assert qg.gemm_run_s8(h, op, p.alpha, qg.ptr(p.a), qg.row_major(p.a), qg.ptr(p.sa), qg.ptr(p.b), qg.col_major_from_nk(p.b), qg.ptr(p.sb), 0.0,
                          None, None, qg.ptr(out), qg.row_major(out), qg.current_stream()) == OK
    assert torch.equal(out.cpu(), p.expected())


def test_mixture_of_experts_as_it_is_used(h):
    """Route, place in int8, experts' up product, quantise, down product, weighted
    sum: captured and replayed, against the same steps in 64 bits."""
    tokens, hidden, inner, experts, topk = 50, 256, 384, 8, 2
    g = torch.Generator().manual_seed(0)
    x = torch.randn(tokens, hidden, generator=g).bfloat16().cuda()
    logits = torch.randn(tokens, experts, generator=g).cuda()
    up_w, down_w = (0.1 * torch.randn(experts, inner, hidden, generator=g)).bfloat16().cuda(), (0.1 * torch.randn(experts, hidden, inner, generator=g)).bfloat16().cuda()
    i8 = lambda *s: torch.zeros(*s, dtype=torch.int8, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    up, up_s, down, down_s = i8(experts, inner, hidden), f32(experts, inner), i8(experts, hidden, inner), f32(experts, hidden)
    ids, w, rows, off = i32(tokens, topk), f32(tokens, topk), i32(tokens, topk), i32(experts + 1)
    n = tokens * topk
    xq, xs, mid, mq, ms, y, out = i8(n, hidden), f32(n), bf(n, inner), i8(n, inner), f32(n), bf(n, hidden), bf(tokens, hidden)
    P, R = qg.ptr, qg.row_major
    route, relu, plain = qg.gemm_route_t(topk=topk, scale=1.0, renormalize=1), qg.gemm_op_t(epilogue=qg.GEMM_EPILOGUE_RELU), qg.gemm_op_t()
    for wt, q, s in ((up_w, up, up_s), (down_w, down, down_s)):
        assert qg.gemm_s8_quantize(h, P(wt), R(wt), P(q), R(q), P(s), qg.current_stream()) == OK

    def step():
        st = qg.current_stream()
        for rc in (qg.gemm_moe_route(h, route, P(logits), R(logits), P(ids), P(w), P(rows), P(off), None, st),
                   qg.gemm_moe_dispatch(h, P(x), R(x), P(rows), topk, P(xq), R(xq), P(xs), st),
                   qg.gemm_run_s8_grouped(h, relu, 1.0, P(xq), R(xq), P(xs), P(up), qg.col_major_from_nk(up), P(up_s), 0.0, None, None, P(mid),
                                          R(mid), P(off), experts, st),
                   qg.gemm_s8_quantize(h, P(mid), R(mid), P(mq), R(mq), P(ms), st),
                   qg.gemm_run_s8_grouped(h, plain, 1.0, P(mq), R(mq), P(ms), P(down), qg.col_major_from_nk(down), P(down_s), 0.0, None, None,
                                          P(y), R(y), P(off), experts, st),
                   qg.gemm_moe_combine(h, P(y), R(y), P(rows), P(w), topk, 1.0, P(x), R(x), P(out), R(out), st)):
            assert rc == OK, qg.gemm_status_string(rc)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        out.zero_()
        logits.copy_(torch.randn(tokens, experts, generator=g))
        graph.replay()
        side.synchronize()
    # each step from what the step before it wrote
    want = ref.route(logits.double().cpu().numpy(), topk)
    assert np.array_equal(ids.cpu().numpy(), want[0]) and np.array_equal(rows.cpu().numpy(), want[2]) and np.array_equal(off.cpu().numpy(), want[3])
    for t in range(tokens):
        q, s = ref.quantize(x[t:t + 1])
        for j in range(topk):
            r = int(rows[t, j])
            assert np.array_equal(xq[r].cpu().numpy(), q[0]) and float(xs[r]) == float(s[0])
    edge = off.tolist()
    for e in range(experts):
        mine = slice(edge[e], edge[e + 1])
        if edge[e + 1] > edge[e]:
            assert torch.equal(mid[mine].cpu(), ref.product(ref.sums(xq[mine], up[e]), 1.0, xs[mine], up_s[e], torch.bfloat16, relu=True))
            assert torch.equal(y[mine].cpu(), ref.product(ref.sums(mq[mine], down[e]), 1.0, ms[mine], down_s[e], torch.bfloat16))
    q, s = ref.quantize(mid)
    assert np.array_equal(mq.cpu().numpy(), q) and np.array_equal(ms.cpu().numpy(), s)
    terms = w.double().cpu().unsqueeze(-1) * y.double().cpu()[rows.long().cpu()]
    full = terms.sum(1) + x.double().cpu()
    tol = 3 * 2.0 ** -24 * (terms.abs().sum(1) + x.double().cpu().abs()) + full.abs() * 2.0 ** -8 * (1 + 2.0 ** -10) + 2.0 ** -25
    assert ((out.double().cpu() - full).abs() <= tol).all()
    assert math.isfinite(float(full.sum()))
