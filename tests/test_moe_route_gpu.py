"""Routing against its definition in 64 bits: the experts chosen, the rows and
the offsets exactly, the weights within fp32's roundings."""
import numpy as np
import pytest
import torch

import moe_ref as ref
import quantized_gemm_tcgen05_gb300 as qg

pytestmark = pytest.mark.gpu
INV, UNS, WSP, OK = qg.GEMM_ERR_INVALID_ARG, qg.GEMM_ERR_UNSUPPORTED, qg.GEMM_ERR_WORKSPACE, qg.GEMM_OK
SCORES = {"softmax": qg.GEMM_ROUTE_SOFTMAX, "sigmoid": qg.GEMM_ROUTE_SIGMOID}


@pytest.fixture(scope="module")
def h():
    h = qg.gemm_create()
    yield h
    qg.gemm_destroy(h)


@pytest.fixture(scope="module")
def ws():
    return qg.Workspace()


def call(h, ws, logits, topk, score="softmax", bias=None, groups=1, group_topk=1, group_best=1, renormalize=True, scale=1.0,
         plan=True, stream=None):
    tokens, experts = logits.shape
    op = qg.gemm_route_t(SCORES[score], topk, groups, group_topk, group_best, int(renormalize), scale, qg.ptr(bias))
    ids = torch.full((tokens, topk), 77, dtype=torch.int32, device="cuda")
    w = torch.full((tokens, topk), 77.0, device="cuda")
    rows = torch.full((tokens, topk), 77, dtype=torch.int32, device="cuda") if plan else None
    off = torch.full((experts + 1,), 77, dtype=torch.int32, device="cuda") if plan else None
    rc = qg.gemm_moe_route(h, op, qg.ptr(logits), qg.row_major(logits), qg.ptr(ids), qg.ptr(w), qg.ptr(rows), qg.ptr(off),
                           ws.c if ws else None, stream or qg.current_stream())
    assert rc == OK, qg.gemm_status_string(rc)
    return ids, w, rows, off


def check(h, ws, logits, topk, **kw):
    got = call(h, ws, logits, topk, **kw)
    bias = kw.get("bias")
    opts = {k: v for k, v in kw.items() if k not in ("bias", "plan")}
    want = ref.route(logits.double().cpu().numpy(), topk, bias=None if bias is None else bias.cpu().numpy(), **opts)
    assert np.array_equal(got[0].cpu().numpy(), want[0])
    if kw.get("plan", True):
        assert np.array_equal(got[2].cpu().numpy(), want[2])
        assert np.array_equal(got[3].cpu().numpy(), want[3])
    w = got[1].double().cpu().numpy()
    assert np.array_equal(np.isnan(w), np.isnan(want[1]))
    l = logits.double().cpu().numpy()
    l = l[np.isfinite(l)]
    spread = float(l.max() - l.min()) if l.size else 0.0
    # two exponentials (2 units each, their arguments rounded: spread * 2^-24), a sum
    # of up to 37 roundings, a quotient, a product: (2 spread + 8 + 40) 2^-24, relative
    tol = (spread + 24) * 2.0 ** -23 * np.abs(want[1]) + 1e-37
    assert np.nanmax(np.abs(w - want[1]) - tol, initial=-1.0) <= 0
    return got


def normal(seed, *shape, x="f32"):
    g = torch.Generator().manual_seed(seed)
    return (1.5 * torch.randn(*shape, generator=g)).to(ref.TORCH[x]).cuda()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tokens,experts,topk", [(1, 1, 1), (1, 8, 2), (16, 8, 8), (64, 64, 6), (65, 33, 5), (300, 256, 8),
                                                 (700, 60, 4), (9, 1000, 32), (2500, 16, 1)])
def test_choice_without_bias(h, ws, tokens, experts, topk, x, score):
    check(h, ws, normal(tokens, tokens, experts, x=x), topk, score=score, renormalize=tokens % 2 == 0, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,experts,topk,groups,keep,best", [
    (33, 8, 2, 1, 1, 1), (400, 256, 8, 8, 4, 2), (150, 160, 6, 8, 3, 1), (70, 64, 8, 32, 16, 2), (40, 12, 3, 4, 1, 2), (31, 6, 4, 6, 2, 2),
    (50, 1024, 8, 16, 4, 2)])
def test_bias_and_groups(h, ws, tokens, experts, topk, groups, keep, best, x, score):
    l = normal(tokens, tokens, experts, x=x)
    bias = (0.1 * torch.randn(experts, generator=torch.Generator().manual_seed(7))).cuda()
    check(h, ws, l, topk, score=score, bias=bias, groups=groups, group_topk=keep, group_best=best)
    if groups > 1:
        check(h, ws, l, topk, score=score, groups=groups, group_topk=keep, group_best=best, renormalize=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(h, ws, score):
    l = torch.zeros(20, 40, device="cuda")
    check(h, ws, l, 7, score=score)
    l[:, 11] = -0.0  # equal to 0
    l[3, 30:] = 1.0
    check(h, ws, l, 7, score=score)
    zero = torch.zeros(40, device="cuda")
    check(h, ws, l, 7, score=score, bias=zero)
    check(h, ws, l, 7, score=score, bias=zero, groups=8, group_topk=2, group_best=2)
    check(h, ws, l, 7, score=score, groups=8, group_topk=3, group_best=1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_that_fp32_cannot_tell_apart(h, ws, score):
    """Biased scores nearer to each other than fp32's error: the order is that of 64
    bits.  A bias of s0 - s_e, rounded to fp32, makes every c nearly equal."""
    experts = 48
    l = normal(1, 30, experts)
    l[:] = l[0]
    s = l[0].double().cpu()
    s = torch.softmax(s, 0) if score == "softmax" else torch.sigmoid(s)
    bias = (s[0] - s).float().cuda()
    c = s + bias.double().cpu()
    assert float(c.max() - c.min()) < 1e-7 and len(set(c.tolist())) > 40
    check(h, ws, l, 8, score=score, bias=bias)
    check(h, ws, l, 8, score=score, bias=bias, groups=12, group_topk=3, group_best=2)
    check(h, ws, l, 8, score=score, bias=bias, groups=12, group_topk=5, group_best=1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("tokens", [20, 200])
def test_masked_experts_and_undefined_tokens(h, ws, tokens, biased, score):
    experts = 24
    l = normal(5, tokens, experts)
    g = torch.Generator().manual_seed(9)
    l[(torch.rand(tokens, experts, generator=g) < 0.8).cuda()] = -torch.inf  # often fewer than topk are left
    l[4] = -torch.inf
    l[5, 3] = torch.nan
    l[6, 2] = torch.inf  # undefined under softmax, a score of 1 under sigmoid
    l[7] = torch.finfo(torch.float32).min  # not masked
    l[8] = torch.finfo(torch.float32).max
    bias = (0.1 * torch.randn(experts, generator=g)).cuda() if biased else None
    if biased:
        bias[10] = -torch.inf
    ids, w, rows, off = check(h, ws, l, 6, score=score, bias=bias)
    assert (ids[4] == -1).all() and (w[4] == 0).all() and (rows[4] == -1).all()
    assert (ids[5] == -1).all() and w[5].isnan().all() and (rows[5] == -1).all()
    check(h, ws, l, 6, score=score, bias=bias, groups=4, group_topk=2, group_best=2)
    if biased:
        bias[3] = torch.nan
        ids, w, rows, off = check(h, ws, l, 6, score=score, bias=bias)
        assert w.isnan().all() and int(off[-1]) == 0


@pytest.mark.parametrize("tokens", [17, 40, 64])
def test_one_block_without_a_workspace(h, ws, tokens):
    l = normal(tokens, tokens, 40)
    bias = (0.1 * torch.randn(40, generator=torch.Generator().manual_seed(3))).cuda()
    for a, b in zip(check(h, None, l, 5, bias=bias), check(h, ws, l, 5, bias=bias)):
        assert torch.equal(a, b)
    bias.fill_(-torch.inf)  # nobody may be chosen
    ids, w, rows, off = check(h, None, l, 5, bias=bias)
    assert (ids == -1).all() and (w == 0).all() and (off == 0).all()


def test_renormalised_weights_of_tiny_scores(h, ws):
    """A bias can choose experts whose scores underflow: their shares are still right."""
    l = torch.zeros(3, 8, device="cuda")
    l[:, 2], l[:, 5] = -150.0, -151.0
    bias = torch.zeros(8, device="cuda")
    bias[2], bias[5] = 4.0, 3.0
    for score in SCORES:
        ids, w, _, _ = check(h, ws, l, 2, score=score, bias=bias)
        assert ids.tolist() == [[2, 5]] * 3


@pytest.mark.parametrize("tokens,experts", [(6000, 1), (6000, 2), (3000, 9), (4000, 257)])
def test_workspace_of_the_stated_size(h, tokens, experts):
    """Nothing past GEMM_ROUTE_SCRATCH bytes is written."""
    n = qg.gemm_route_scratch(experts)
    buf = torch.full((n + 65536,), 171, dtype=torch.uint8, device="cuda")

    class Exact:
        c = qg.gemm_workspace_t(None, 0, qg.ptr(buf), n)

    check(h, Exact, normal(1, tokens, experts, x="bf16"), 1)
    assert (buf[n:] == 171).all()


def test_no_tokens(h, ws):
    l = torch.empty(0, 8, device="cuda")
    off = torch.full((9,), 5, dtype=torch.int32, device="cuda")
    op = qg.gemm_route_t(topk=2, scale=1.0)
    assert qg.gemm_moe_route(h, op, None, qg.row_major(l), None, None, None, qg.ptr(off), None, qg.current_stream()) == OK
    assert off.tolist() == [0] * 9
    assert qg.gemm_moe_route(h, op, None, qg.row_major(l), None, None, None, None, None, qg.current_stream()) == OK


@pytest.mark.parametrize("tokens", [7, 900])
def test_strides_and_choice_alone(h, ws, tokens):
    wide = normal(3, tokens, 50)
    check(h, ws, wide[:, 3:40], 5, plan=False)
    check(h, None, wide[:, 3:40], 5, plan=False)  # no plan, no workspace
    check(h, ws, wide[:, 3:40], 5)


def test_long_prompt(h, ws):
    """More tokens than one a warp: many tokens a block, and offsets that add up."""
    check(h, ws, normal(2, 6000, 8, x="bf16"), 2)
    ids, w, rows, off = call(h, ws, normal(4, 70000, 128, x="bf16"), 4)
    n = torch.bincount(ids.reshape(-1).long(), minlength=128)
    assert torch.equal(off[1:].long(), n.cumsum(0))
    flat = ids.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    assert torch.equal(rows.reshape(-1)[order].long(), torch.arange(flat.numel(), device="cuda"))


def test_graphs_share_a_workspace_and_streams(h, ws):
    """Captured and replayed on another stream; two graphs that share the workspace run one after another."""
    l1, l2 = normal(1, 300, 32), normal(2, 500, 64)
    side = torch.cuda.Stream()
    outs, graphs = [], []
    with torch.cuda.stream(side):
        for l in (l1, l2):
            call(h, ws, l, 3)
            side.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                op = qg.gemm_route_t(topk=3, scale=1.0, renormalize=1)
                o = [torch.empty(l.shape[0], 3, dtype=torch.int32, device="cuda"), torch.empty(l.shape[0], 3, device="cuda"),
                     torch.empty(l.shape[0], 3, dtype=torch.int32, device="cuda"), torch.empty(l.shape[1] + 1, dtype=torch.int32, device="cuda")]
                assert qg.gemm_moe_route(h, op, qg.ptr(l), qg.row_major(l), *[qg.ptr(t) for t in o], ws.c, qg.current_stream()) == OK
            graphs.append(g)
            outs.append(o)
        for _ in range(3):
            for g in graphs:
                g.replay()
        l1.copy_(normal(8, 300, 32))
        for g in graphs:
            g.replay()
        side.synchronize()
    for l, o in zip((l1, l2), outs):
        want = ref.route(l.double().cpu().numpy(), 3)
        for i in (0, 2, 3):
            assert np.array_equal(o[i].cpu().numpy(), want[i])


def test_refusals(h, ws):
    l = normal(1, 100, 16)
    ids, w = torch.full((100, 4), 9, dtype=torch.int32, device="cuda"), torch.full((100, 4), 9.0, device="cuda")
    rows, off = torch.full_like(ids, 9), torch.full((17,), 9, dtype=torch.int32, device="cuda")
    bias = torch.zeros(16, device="cuda")
    host = torch.zeros(4096)
    base = dict(score=0, topk=4, groups=0, group_topk=0, group_best=0, renormalize=1, scale=1.0, bias=None)
    arg = dict(L=qg.ptr(l), Ldesc=qg.row_major(l), ids=qg.ptr(ids), weights=qg.ptr(w), rows=qg.ptr(rows), expert_offsets=qg.ptr(off),
               workspace=ws.c)
    lay = lambda **kw: qg.gemm_layout_t(**{**{f: getattr(arg["Ldesc"], f) for f, _ in qg.gemm_layout_t._fields_}, **kw})  # noqa: E731
    small = qg.gemm_workspace_t(None, 0, ws.c.partials, qg.gemm_route_scratch(16) - 1)
    assert qg.gemm_route_scratch(16) == 304 * 32 and qg.gemm_route_scratch(1) == 304 * 16
    cases = [
        (dict(score=2), {}, UNS), (dict(score=-1), {}, UNS), (dict(topk=0), {}, INV), (dict(topk=17), {}, INV), (dict(scale=float("nan")), {}, INV),
        (dict(scale=float("inf")), {}, INV), (dict(renormalize=2), {}, INV), (dict(groups=-1), {}, INV),
        (dict(groups=3, group_topk=1, group_best=1), {}, INV), (dict(groups=4, group_topk=0, group_best=1), {}, INV),
        (dict(groups=4, group_topk=5, group_best=1), {}, INV), (dict(groups=4, group_topk=1, group_best=3), {}, INV),
        (dict(groups=4, group_topk=1, group_best=0), {}, INV),
        (dict(bias=host.data_ptr()), {}, INV), (dict(bias=qg.ptr(bias) + 2), {}, INV),
        ({}, dict(L=None), INV), ({}, dict(L=host.data_ptr()), INV), ({}, dict(L=arg["L"] + 2), INV), ({}, dict(Ldesc=None), INV),
        ({}, dict(ids=None), INV), ({}, dict(weights=None), INV), ({}, dict(weights=arg["weights"] + 1), INV),
        ({}, dict(rows=None), INV), ({}, dict(expert_offsets=None), INV), ({}, dict(expert_offsets=host.data_ptr()), INV),
        ({}, dict(workspace=None), WSP), ({}, dict(workspace=small), WSP),
        ({}, dict(workspace=qg.gemm_workspace_t(None, 0, host.data_ptr(), 1 << 20)), INV),
        ({}, dict(Ldesc=lay(type=qg.GEMM_E4M3)), UNS), ({}, dict(Ldesc=lay(order=1)), UNS), ({}, dict(Ldesc=lay(ld=15)), INV),
        ({}, dict(Ldesc=lay(num=2)), UNS), ({}, dict(Ldesc=lay(cols=1025, ld=1025)), UNS), ({}, dict(Ldesc=lay(cols=0)), INV),
        ({}, dict(Ldesc=lay(rows=-1)), INV), ({}, dict(Ldesc=lay(rows=1 << 30)), UNS),
    ]
    for o, a, want in cases:
        rc = qg.gemm_moe_route(h, qg.gemm_route_t(**{**base, **o}), *({**arg, **a}).values(), qg.current_stream())
        assert rc == want, (o, a, rc)
    big = normal(1, 4, 1024)
    op = qg.gemm_route_t(**{**base, "topk": 33})
    assert qg.gemm_moe_route(h, op, qg.ptr(big), qg.row_major(big), *[arg[k] for k in ("ids", "weights", "rows", "expert_offsets", "workspace")],
                             qg.current_stream()) == UNS
    op = qg.gemm_route_t(**{**base, "groups": 64, "group_topk": 1, "group_best": 1})
    assert qg.gemm_moe_route(h, op, qg.ptr(big), qg.row_major(big), *[arg[k] for k in ("ids", "weights", "rows", "expert_offsets", "workspace")],
                             qg.current_stream()) == UNS
    assert qg.gemm_moe_route(h, None, *arg.values(), qg.current_stream()) == INV
    torch.cuda.synchronize()
    assert (ids == 9).all() and (w == 9).all() and (rows == 9).all() and (off == 9).all()
