"""Performance cases of the operators of an 8-bit mixture of experts: routing,
quantisation of token rows to int8 (dense, or while they are placed by expert),
the dense and the grouped int8 product, and the weighted sum that brings the
experts' rows back to their tokens.

Every case has a plain form (elementary torch operations) and the library's own
form, which `run` takes when `own` is set.  Both read the same prepared state.

Definitions.
  Routing.  s = softmax(l) or sigmoid(l) of a token's E logits, c = s + bias.  An
  expert whose logit or bias is -inf is never chosen.  With groups, a group's
  score is the sum of its `best` largest c, and only the `keep` groups with the
  largest scores take part.  The topk experts with the largest c (without a
  bias: with the largest logits) are chosen, in that order; ties go to the
  lowest index.  Weights are the chosen s, divided by their sum where `renorm`
  is set, times a factor.  Which experts are chosen is decided in 64 bits.  A
  slot for which no expert is left has id -1, weight 0, row -1.  Rows: the
  (token, slot) pairs sorted by expert, then by token; offsets: where each
  expert's rows start.
  Quantisation.  amax = max |x| of a row, scale = max(amax / 127, 2^-126),
  code = RN(x * (127 / amax)), every step rounded to fp32.
  Product.  D = act(alpha * sa[i] * sb[j] * sum_k a[i][k] b[j][k] + beta C + bias).
  Weighted sum.  D[t] = beta C[t] + sum_j w[t][j] Y[row[t][j]].
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "s8": 1}


# ---- cases ------------------------------------------------------------------

def _r(name, tokens, experts, topk, x, score, bias, groups=1, keep=1, best=1, renorm=True, masked=False):
    """Route tokens by their logits of type x."""
    return dict(name=name, op="route", tokens=tokens, experts=experts, topk=topk, x=x, score=score, bias=bias, groups=groups, keep=keep, best=best,
                renorm=renorm, masked=masked)


def _q(name, rows, k, x, pad=0):
    """Quantise rows x k values of type x (row stride k + pad) row by row."""
    return dict(name=name, op="quantize", rows=rows, k=k, x=x, pad=pad)


def _d(name, tokens, h, topk, x, to, experts):
    """Place every token's row at its topk rows by expert, as type `to`."""
    return dict(name=name, op="dispatch", tokens=tokens, h=h, topk=topk, x=x, to=to, experts=experts)


def _p(name, m, n, k, d, act="", beta=0.0):
    """D[m, n] = act(alpha sa sb A B^T + beta C + bias), A and B int8."""
    return dict(name=name, op="product", m=m, n=n, k=k, d=d, act=act, beta=beta)


def _g(name, rows, experts, n, k, d):
    """Rows sorted by expert, each times its own expert's n x k matrix."""
    return dict(name=name, op="grouped", rows=rows, experts=experts, n=n, k=k, d=d)


def _c(name, tokens, h, topk, x, beta=0.0, experts=8):
    """Every token's weighted sum of its topk rows."""
    return dict(name=name, op="combine", tokens=tokens, h=h, topk=topk, x=x, beta=beta, experts=experts)


def listed():
    return [
        # sixteen decoding tokens, two of eight experts each: a latency
        _r("route 16x8 top 2", 16, 8, 2, "bf16", "softmax", False),
        # a prompt over many small experts, chosen group by group, with a bias for balance
        _r("route 4001x256 top 8", 4001, 256, 8, "f32", "sigmoid", True, 8, 4, 2),
        # a prompt's activations before a down projection
        _q("quantize 4096x14336", 4096, 14336, "bf16"),
        # sixteen decoding tokens' rows to two experts each, in 8 bits
        _d("dispatch 16x4096 top 2 s8", 16, 4096, 2, "bf16", "s8", 8),
        # a prompt's rows to six experts each, copied; a row length that no vector fits
        _d("dispatch 1333x4104 top 6", 1333, 4104, 6, "f16", "f16", 64),
        # one token through a down projection: the weights are the work
        _p("product 1x4096x14336", 1, 4096, 14336, "bf16"),
        # decoding sequences through an up projection, sizes that fit no tile
        _p("product 77x11002x4104", 77, 11002, 4104, "f16", act="gelu"),
        # the square product that dense throughput is quoted on, added to what is there
        _p("product 4096x4096x4096", 4096, 4096, 4096, "bf16", beta=0.5),
        # sixteen decoding tokens, each routed to two of eight experts
        _g("grouped 32x8x14336x4096", 32, 8, 14336, 4096, "bf16"),
        # a prompt of 4096 routed rows, popular experts first
        _g("grouped 4096x8x14336x4096", 4096, 8, 14336, 4096, "bf16"),
        # sixteen decoding tokens' two experts
        _c("combine 16x4096 top 2", 16, 4096, 2, "bf16"),
        # a prompt's six experts, added to what all tokens share
        _c("combine 4096x4096 top 6", 4096, 4096, 6, "bf16", beta=1.0, experts=64),
    ]


def _log(rng, lo, hi):
    return min(max(int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))), lo), hi)


def draw(rng):
    op = rng.choice(["route", "route", "quantize", "dispatch", "product", "product", "grouped", "combine"])
    x = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "route":
        experts, groups = rng.choice([(8, 1), (8, 1), (16, 1), (60, 1), (64, 8), (128, 1), (160, 8), (256, 8), (256, 8), (384, 1)])
        topk = rng.randint(1, 8)
        keep = rng.randint(max(1, groups // 2), groups)
        c = _r("", _log(rng, 1, 4096), experts, topk, x, rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5, groups, keep,
               rng.choice([1, 2]) if groups > 1 else 1, rng.random() < 0.7, rng.random() < 0.25)
    elif op == "quantize":
        c = _q("", _log(rng, 1, 4096), _log(rng, 64, 14336), x, rng.choice([0, 0, 8, 3]))
    elif op == "dispatch":
        c = _d("", _log(rng, 1, 4096), _log(rng, 64, 8192), rng.randint(1, 8), x, rng.choice(["s8", "s8", x]), rng.choice([8, 64]))
    elif op == "product":
        # rows of codes start every 16 bytes; K need not be a multiple of that
        c = _p("", _log(rng, 1, 4096), _log(rng, 64, 14336), _log(rng, 64, 4096), x, rng.choice(["", "", "gelu", "relu"]),
               rng.choice([0.0, 0.0, 0.5]))
    elif op == "grouped":
        c = _g("", _log(rng, 4, 4096), rng.choice([2, 8, 8, 32]), _log(rng, 64, 4096), _log(rng, 64, 4096), x)
    else:
        c = _c("", _log(rng, 1, 4096), _log(rng, 64, 8192), rng.randint(1, 8), x, rng.choice([0.0, 1.0]), rng.choice([8, 64]))
    del c["name"]
    return c


# ---- inputs -----------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _activations(gen, rows, k):
    """Normal values with a few loud channels, as hidden states have them."""
    loud = torch.where(torch.rand(k, generator=gen, device="cuda") < 0.01, 12.0, 1.0)
    return _normal(gen, rows, k) * loud


def _popularity(gen, experts):
    """How often experts are wanted: falls off as 1 / rank^1.2."""
    p = torch.arange(1, experts + 1, device="cuda", dtype=torch.float64) ** -1.2
    return p[torch.randperm(experts, generator=gen, device="cuda")]


def _offsets_of(pick, experts):
    count = torch.bincount(pick, minlength=experts)
    return torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(count, 0)]).int()


def _placed(ids, experts):
    """Rows of (token, slot) pairs sorted by expert, then by token; ids of -1 have none."""
    flat = torch.where(ids < 0, experts, ids).reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    rows = torch.empty_like(flat)
    rows[order] = torch.arange(flat.numel(), device=flat.device)
    return torch.where(flat < experts, rows, -1).int().view(ids.shape)


def _routed(gen, tokens, experts, topk):
    """The rows that a routing of these tokens would give."""
    wanted = _popularity(gen, experts).log() - torch.log(-torch.log(torch.rand(tokens, experts, generator=gen, device="cuda").double()))
    ids = torch.argsort(wanted, dim=1, descending=True)[:, :topk]
    return _placed(ids, experts)


def _codes(x):
    """int8 rows that start every 16 bytes, and one scale each."""
    amax = x.abs().amax(-1, keepdim=True).clamp(min=1e-30)
    full = torch.zeros(*x.shape[:-1], -(-x.shape[-1] // 16) * 16, dtype=torch.int8, device=x.device)
    full[..., :x.shape[-1]] = torch.round(x * (127.0 / amax)).to(torch.int8)
    return full[..., :x.shape[-1]], (amax / 127.0).squeeze(-1).contiguous()


def prepare(case, seed):
    gen, s = _gen(seed), dict(case)
    op = case["op"]
    new = lambda *shape, dtype: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    if op == "route":
        tokens, experts, topk = case["tokens"], case["experts"], case["topk"]
        logits = 1.5 * _normal(gen, tokens, experts) + 0.5 * _normal(gen, experts)
        if case["masked"]:
            logits[torch.rand(tokens, experts, generator=gen, device="cuda") < 0.5] = -math.inf
            logits[torch.rand(tokens, generator=gen, device="cuda") < 0.1] = -math.inf
        s["logits"] = logits.to(TYPES[case["x"]])
        s["bias_values"] = 0.1 * _normal(gen, experts) if case["bias"] else None
        s["factor"] = 2.5 if case["score"] == "sigmoid" else 1.0
        s["ids"], s["rows_out"] = new(tokens, topk, dtype=torch.int32), new(tokens, topk, dtype=torch.int32)
        s["weights"], s["offsets"] = new(tokens, topk, dtype=torch.float32), new(experts + 1, dtype=torch.int32)
        s["scratch"] = torch.zeros(4 << 20, dtype=torch.uint8, device="cuda")
    elif op == "quantize":
        rows, k = case["rows"], case["k"]
        s["x_values"] = _activations(gen, rows, k + case["pad"]).to(TYPES[case["x"]])[:, :k]
        s["codes"], s["scales"] = new(rows, k, dtype=torch.int8), new(rows, dtype=torch.float32)
    elif op == "dispatch":
        tokens, h, topk = case["tokens"], case["h"], case["topk"]
        s["x_values"] = _activations(gen, tokens, h).to(TYPES[case["x"]])
        s["rows_of"] = _routed(gen, tokens, case["experts"], topk)
        s["placed"] = new(tokens * topk, h, dtype=torch.int8 if case["to"] == "s8" else TYPES[case["to"]])
        s["scales"] = new(tokens * topk, dtype=torch.float32) if case["to"] == "s8" else None
    elif op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["sa"] = _codes(_activations(gen, m, k))
        s["b"], s["sb"] = _codes(0.02 * _normal(gen, n, k))
        s["alpha"] = 1.5
        s["c"] = _normal(gen, m, n).to(TYPES[case["d"]]) if case["beta"] else None
        s["bias"] = _normal(gen, n).to(torch.bfloat16) if case["act"] else None
        s["out"] = torch.empty(m, n, dtype=TYPES[case["d"]], device="cuda")
    elif op == "grouped":
        rows, experts, n, k = case["rows"], case["experts"], case["n"], case["k"]
        s["offsets"] = _offsets_of(torch.multinomial(_popularity(gen, experts), rows, replacement=True, generator=gen), experts)
        s["host_offsets"] = s["offsets"].tolist()  # the plain form cuts its products on the host
        s["a"], s["sa"] = _codes(_activations(gen, rows, k))
        w = [_codes(0.02 * _normal(gen, n, k)) for _ in range(experts)]
        full = new(experts, n, -(-k // 16) * 16, dtype=torch.int8)
        for e in range(experts):
            full[e, :, :k] = w[e][0]
        s["b"], s["sb"] = full[:, :, :k], torch.stack([v[1] for v in w])
        s["out"] = torch.empty(rows, n, dtype=TYPES[case["d"]], device="cuda")
    else:
        tokens, h, topk, x = case["tokens"], case["h"], case["topk"], TYPES[case["x"]]
        s["rows_of"] = _routed(gen, tokens, case["experts"], topk)
        s["y"] = _normal(gen, tokens * topk, h).to(x)
        w = torch.rand(tokens, topk, generator=gen, device="cuda") + 0.05
        s["w"] = w / w.sum(1, keepdim=True)
        s["c"] = _normal(gen, tokens, h).to(x) if case["beta"] else None
        s["out"] = torch.empty(tokens, h, dtype=x, device="cuda")
    return s


# ---- one pass, plain --------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _quantized(x):
    v = x.float()
    amax = v.abs().amax(-1, keepdim=True)
    # a tensor divides; a Python number would be turned into a factor
    top = torch.full((1,), 127.0, dtype=torch.float32, device=x.device)
    scale = torch.clamp(amax / top, min=2.0 ** -126)
    factor = torch.where(amax / top >= 2.0 ** -126, top / amax, 2.0 ** 126)
    return torch.round(v * factor).to(torch.int8), scale.squeeze(-1)


def _sums(a, b):
    """a b^T of int8 codes: fp32 holds the sums of 1024 products exactly, longer
    ones are added up in 64 bits."""
    k = a.shape[-1]
    if k <= 1024:
        return a.float() @ b.float().t()
    parts = -(-k // 1024)
    fill = parts * 1024 - k
    a = torch.nn.functional.pad(a.float(), (0, fill)).view(a.shape[0], parts, 1024).transpose(0, 1)
    b = torch.nn.functional.pad(b.float(), (0, fill)).view(b.shape[0], parts, 1024).transpose(0, 1)
    return torch.bmm(a, b.transpose(1, 2)).sum(0, dtype=torch.float64).float()


def _finish(acc, s):
    """Scales, C, bias and activation in fp32, one rounding."""
    y = acc * (s["alpha"] * s["sa"])[:, None] * s["sb"]
    if s["c"] is not None:
        y = y + s["beta"] * s["c"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if s["act"] == "relu":
        y = torch.where(y < 0, 0.0, y)
    if s["act"] == "gelu":
        y = 0.5 * y * torch.erfc(y * -0.7071067811865476)
    return y.to(TYPES[s["d"]])


def _run_plain(s):
    op = s["op"]
    if op == "route":
        return _route(s)
    if op == "quantize":
        codes, scales = _quantized(s["x_values"])
        return {"codes": codes, "scales": scales}
    if op == "dispatch":
        at = s["rows_of"].reshape(-1).long()
        x = s["x_values"]
        placed = torch.zeros_like(s["placed"])
        if s["to"] != "s8":
            placed[at] = x.repeat_interleave(s["topk"], 0)
            return {"placed": placed}
        codes, scale = _quantized(x)
        scales = torch.zeros_like(s["scales"])
        placed[at] = codes.repeat_interleave(s["topk"], 0)
        scales[at] = scale.repeat_interleave(s["topk"], 0)
        return {"placed": placed, "scales": scales}
    if op == "product":
        return _finish(_sums(s["a"], s["b"]), s)
    if op == "grouped":
        off = s["host_offsets"]
        y = torch.empty(s["rows"], s["n"], dtype=torch.float32, device=s["a"].device)
        # one product per expert that has rows: cutting here is cheaper than
        # padding every expert to the most popular one's rows
        for e in range(s["experts"]):
            if off[e + 1] > off[e]:
                mine = slice(off[e], off[e + 1])
                y[mine] = _sums(s["a"][mine], s["b"][e]) * s["sa"][mine, None] * s["sb"][e]
        return y.to(TYPES[s["d"]])
    y = (s["y"].float()[s["rows_of"].long()] * s["w"][:, :, None]).sum(1)
    if s["c"] is not None:
        y = y + s["beta"] * s["c"].float()
    return y.to(TYPES[s["x"]])


def _route(s):
    """In 64 bits: scores next to a border decide whole numbers."""
    l = s["logits"].double()
    tokens, experts = l.shape
    live = l > -math.inf
    if s["score"] == "softmax":
        top = l.amax(1, keepdim=True)
        e = torch.exp(l - torch.where(top > -math.inf, top, 0.0))
        total = e.sum(1, keepdim=True)
        p = e / torch.where(total > 0, total, 1.0)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    c = p if s["bias_values"] is None else p + s["bias_values"].double()
    c = torch.where(live, c, -math.inf)
    key = torch.where(live, l, -math.inf) if s["bias_values"] is None else c
    if s["groups"] > 1:
        best = c.view(tokens, s["groups"], -1).sort(2, descending=True).values[:, :, :s["best"]]
        none = best[:, :, 0] == -math.inf
        score = torch.where(none, -math.inf, torch.where(best > -math.inf, best, 0.0).sum(2))
        taken = score.sort(dim=1, descending=True, stable=True).indices[:, :s["keep"]]
        kept = torch.zeros(tokens, s["groups"], dtype=torch.bool, device=l.device).scatter_(1, taken, True)
        key = torch.where(kept.repeat_interleave(experts // s["groups"], 1), key, -math.inf)
    key, ids = key.sort(dim=1, descending=True, stable=True)
    key, ids = key[:, :s["topk"]], ids[:, :s["topk"]]
    chosen = key > -math.inf
    w = torch.where(chosen, p.gather(1, ids), 0.0)
    if s["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    ids = torch.where(chosen, ids, -1).int()
    count = torch.zeros(experts + 1, dtype=torch.int64, device=l.device)
    count.index_add_(0, torch.where(chosen, ids.long() + 1, 0).reshape(-1), chosen.reshape(-1).long())
    return {"ids": ids, "weights": (w * s["factor"]).float(), "rows": _placed(ids, experts), "offsets": torch.cumsum(count, 0).int()}


# ---- one pass, the library's ------------------------------------------------

_handle = None


def _plan(qg, s):
    """The call and the descriptors that a program keeps beside its buffers."""
    global _handle
    if _handle is None:
        _handle = qg.gemm_create()
    h, op = _handle, s["op"]
    mat = lambda t: None if t is None else qg.row_major(t)  # noqa: E731
    if op == "route":
        o = qg.gemm_route_t(score={"softmax": qg.GEMM_ROUTE_SOFTMAX, "sigmoid": qg.GEMM_ROUTE_SIGMOID}[s["score"]], topk=s["topk"],
                            groups=s["groups"], group_topk=s["keep"], group_best=s["best"], renormalize=int(s["renorm"]), scale=s["factor"],
                            bias=qg.ptr(s["bias_values"]))
        ws = qg.gemm_workspace_t(None, 0, qg.ptr(s["scratch"]), s["scratch"].numel())
        return (qg.gemm_moe_route, (h, o, qg.ptr(s["logits"]), mat(s["logits"]), qg.ptr(s["ids"]), qg.ptr(s["weights"]), qg.ptr(s["rows_out"]),
                                    qg.ptr(s["offsets"]), ws),
                {"ids": s["ids"], "weights": s["weights"], "rows": s["rows_out"], "offsets": s["offsets"]})
    if op == "quantize":
        return (qg.gemm_s8_quantize, (h, qg.ptr(s["x_values"]), mat(s["x_values"]), qg.ptr(s["codes"]), mat(s["codes"]), qg.ptr(s["scales"])),
                {"codes": s["codes"], "scales": s["scales"]})
    if op == "dispatch":
        out = {"placed": s["placed"]} if s["scales"] is None else {"placed": s["placed"], "scales": s["scales"]}
        return (qg.gemm_moe_dispatch, (h, qg.ptr(s["x_values"]), mat(s["x_values"]), qg.ptr(s["rows_of"]), s["topk"], qg.ptr(s["placed"]),
                                       mat(s["placed"]), qg.ptr(s["scales"])), out)
    if op == "combine":
        return (qg.gemm_moe_combine, (h, qg.ptr(s["y"]), mat(s["y"]), qg.ptr(s["rows_of"]), qg.ptr(s["w"]), s["topk"], s["beta"], qg.ptr(s["c"]),
                                      mat(s["c"]), qg.ptr(s["out"]), mat(s["out"])), s["out"])
    o = qg.gemm_op_t()
    a, b, out = (qg.ptr(s["a"]), mat(s["a"]), qg.ptr(s["sa"])), (qg.ptr(s["b"]), qg.col_major_from_nk(s["b"]), qg.ptr(s["sb"])), s["out"]
    if op == "grouped":
        return (qg.gemm_run_s8_grouped, (h, o, 1.0, *a, *b, 0.0, None, None, qg.ptr(out), mat(out), qg.ptr(s["offsets"]), s["experts"]), out)
    if s["bias"] is not None:
        o.epilogue = qg.GEMM_EPILOGUE_BIAS | {"gelu": qg.GEMM_EPILOGUE_GELU, "relu": qg.GEMM_EPILOGUE_RELU}[s["act"]]
        o.bias, o.bias_type = qg.ptr(s["bias"]), qg.GEMM_BF16
    return (qg.gemm_run_s8, (h, o, s["alpha"], *a, *b, s["beta"], qg.ptr(s["c"]), mat(s["c"]), qg.ptr(out), mat(out)), out)


def _run_own(s):
    import quantized_gemm_tcgen05_gb300 as qg

    if "plan" not in s:
        s["plan"] = _plan(qg, s)
    call, args, out = s["plan"]
    rc = call(*args, qg.current_stream())
    if rc:
        raise qg.GemmError(rc, call.__name__)
    return out


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    op = case["op"]
    if op == "route":
        tokens, experts, topk = case["tokens"], case["experts"], case["topk"]
        return {"bytes": tokens * experts * SIZE[case["x"]] + 12 * tokens * topk + 4 * (experts + 1) + (4 * experts if case["bias"] else 0),
                "flops": 4 * tokens * experts}
    if op == "quantize":
        rows, k = case["rows"], case["k"]
        return {"bytes": rows * k * (SIZE[case["x"]] + 1) + 4 * rows, "flops": 3 * rows * k}
    if op == "dispatch":
        tokens, h, topk = case["tokens"], case["h"], case["topk"]
        out = h * SIZE[case["to"]] + (4 if case["to"] == "s8" else 0)
        return {"bytes": tokens * (h * SIZE[case["x"]] + topk * (out + 4)), "flops": 3 * tokens * h if case["to"] == "s8" else 0}
    if op == "product":
        m, n, k, d = case["m"], case["n"], case["k"], SIZE[case["d"]]
        return {"bytes": m * k + n * k + 4 * (m + n) + m * n * d * (2 if case["beta"] else 1), "flops": 2 * m * n * k}
    if op == "grouped":
        rows, n, k = case["rows"], case["n"], case["k"]
        # the experts that 1 / rank^1.2 popularity is expected to give rows
        p = [i ** -1.2 for i in range(1, case["experts"] + 1)]
        met = sum(1.0 - (1.0 - v / sum(p)) ** rows for v in p)
        return {"bytes": rows * (k + 4) + met * n * (k + 4) + rows * n * SIZE[case["d"]], "flops": 2 * rows * n * k}
    tokens, h, topk, x = case["tokens"], case["h"], case["topk"], SIZE[case["x"]]
    return {"bytes": tokens * h * x * (topk + (2 if case["beta"] else 1)) + 8 * tokens * topk, "flops": 2 * tokens * topk * h}


# ---- the definitions in 64 bits ---------------------------------------------

def _exact_codes(x):
    """Every step of the definition, rounded to fp32 from 64 bits."""
    x = x.double()
    amax = x.abs().amax(1)
    scale = (amax / torch.full_like(amax, 127.0)).float().double()
    factor = (torch.full_like(amax, 127.0) / torch.where(amax > 0, amax, 1.0)).float().double()
    tiny = scale < 2.0 ** -126
    scale, factor = torch.where(tiny, 2.0 ** -126, scale), torch.where(tiny, 2.0 ** 126, factor)
    return torch.round((x * factor[:, None]).float()).to(torch.int8), scale


def _exact_route(s):
    """Choice by choice: the largest that is left, the lowest index of equals."""
    l, experts, topk = s["logits"].double(), s["experts"], s["topk"]
    tokens = l.shape[0]
    index = torch.arange(experts, device=l.device)
    dead = torch.isneginf(l)
    if s["score"] == "softmax":
        p = torch.where(dead, 0.0, torch.exp(l - torch.logsumexp(l, 1, keepdim=True)))
    else:
        p = torch.where(dead, 0.0, torch.sigmoid(l))
    biased = s["bias_values"] is not None
    c = torch.where(dead, -math.inf, p + (s["bias_values"].double() if biased else 0.0))

    def largest(v):
        """(value, index) of the largest of every row, the lowest index of equals."""
        top = v.amax(1)
        return top, torch.where(v == top[:, None], torch.arange(v.shape[1], device=v.device), v.shape[1]).amin(1)

    allowed = torch.ones_like(dead)
    if s["groups"] > 1:
        size = experts // s["groups"]
        left, total = c.clone(), torch.zeros(tokens, s["groups"], dtype=torch.float64, device=l.device)
        for i in range(s["best"]):
            for g in range(s["groups"]):
                top, at = largest(left[:, g * size:(g + 1) * size])
                total[:, g] += torch.where(top > -math.inf, top, 0.0)
                left[torch.arange(tokens, device=l.device), g * size + at] = -math.inf
        any_live = (c.view(tokens, s["groups"], size) > -math.inf).any(2)
        total = torch.where(any_live, total, -math.inf)
        taken = torch.zeros(tokens, s["groups"], dtype=torch.bool, device=l.device)
        for i in range(s["keep"]):
            _, at = largest(total)
            taken[torch.arange(tokens, device=l.device), at] = True
            total[torch.arange(tokens, device=l.device), at] = -math.inf
        allowed = taken[:, index // size]
    key = torch.where(allowed & ~dead, c if biased else l, -math.inf)
    ids = torch.full((tokens, topk), -1, dtype=torch.int32, device=l.device)
    w = torch.zeros(tokens, topk, dtype=torch.float64, device=l.device)
    row = torch.arange(tokens, device=l.device)
    for j in range(min(topk, experts)):
        top, at = largest(key)
        have = top > -math.inf
        ids[:, j] = torch.where(have, at, -1).int()
        w[:, j] = torch.where(have, p[row, at], 0.0)
        key[row, at] = -math.inf
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    match = (ids.reshape(-1, 1) == index).long()
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=l.device)
    offsets[1:] = match.sum(0).cumsum(0)
    before = match.cumsum(0) - match
    rows = torch.where(ids.reshape(-1) >= 0, ((before + offsets[:-1]) * match).sum(1), -1)
    return {"ids": ids, "weights": w * s["factor"], "rows": rows.int().view(tokens, topk), "offsets": offsets.int()}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "quantize":
        codes, scales = _exact_codes(s["x_values"])
        return {"codes": codes, "scales": scales}
    if op == "dispatch":
        at = s["rows_of"].long()
        token = torch.empty(at.numel(), dtype=torch.int64, device=at.device)
        token[at.reshape(-1)] = torch.arange(at.numel(), device=at.device) // case["topk"]
        if case["to"] != "s8":
            return {"placed": s["x_values"].double()[token]}
        codes, scales = _exact_codes(s["x_values"])
        return {"placed": codes[token], "scales": scales[token]}
    if op == "product":
        y = s["alpha"] * (s["a"].double() * s["sa"].double()[:, None]) @ (s["b"].double() * s["sb"].double()[:, None]).t()
        if case["beta"]:
            y += case["beta"] * s["c"].double()
        if case["act"]:
            y += s["bias"].double()
            y = torch.clamp(y, min=0.0) if case["act"] == "relu" else y * torch.special.ndtr(y)
        return y
    if op == "grouped":
        off = s["offsets"].tolist()
        return torch.cat([(s["a"][off[e]:off[e + 1]].double() * s["sa"][off[e]:off[e + 1], None].double()) @
                          (s["b"][e].double() * s["sb"][e][:, None].double()).t() for e in range(case["experts"])])
    y = case["beta"] * s["c"].double() if case["beta"] else torch.zeros(case["tokens"], case["h"], dtype=torch.float64, device="cuda")
    for j in range(case["topk"]):
        y = y + s["w"][:, j:j + 1].double() * s["y"][s["rows_of"][:, j].long()].double()
    return y
