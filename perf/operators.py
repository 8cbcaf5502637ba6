"""Performance cases of the 4-bit microscaled operators: quantisation, the
dense and the grouped product, and the residual norm that writes its result in
4 bits.

Every case has a plain form (elementary torch operations in 32 bits) and the
library's own form, which `run` takes when `own` is set.  Both read the same
prepared state.

Formats.  A value is an E2M1 code times its block's scale times the tensor's
scale g.  "nvfp4": blocks of 16 along K, E4M3 scales
s = RN(min(amax / (6 g), 448)); "mxfp4": blocks of 32, scales
2^(floor(log2 amax) - 2) stored as E8M0, g = 1.  A code is RN_E2M1(x / (s g)),
ties to even, saturating at 6 (0 where s = 0); every intermediate value is
rounded to fp32.  Codes are packed two per byte, even k in the low bits.
Scales are stored in 512-byte atoms of 128 rows x 4 blocks: byte
(r % 32) * 16 + (r / 32) * 4 + j, atoms along K first, zero where padded.  Rows
sorted by expert start every expert on an atom row of its own.
"""
import math

import torch

own = False

NV, MX = "nvfp4", "mxfp4"
BLOCK = {NV: 16, MX: 32}
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SCALE_TYPE = {NV: torch.float8_e4m3fn, MX: torch.float8_e8m0fnu}


# ---- cases ------------------------------------------------------------------

def _q(name, rows, k, x, fmt, experts=0, pad=0, g=1.0):
    """Quantise rows x k values of type x (row stride k + pad)."""
    return dict(name=name, op="quantize", rows=rows, k=k, x=x, fmt=fmt, experts=experts, pad=pad, g=g)


def _p(name, m, n, k, d, fmt, act="", beta=0.0):
    """D[m, n] = act(alpha A B^T + beta C + bias), A and B in 4 bits."""
    return dict(name=name, op="product", m=m, n=n, k=k, d=d, fmt=fmt, act=act, beta=beta)


def _g(name, rows, experts, n, k, d, fmt):
    """Rows sorted by expert, each times its own expert's n x k matrix."""
    return dict(name=name, op="grouped", rows=rows, experts=experts, n=n, k=k, d=d, fmt=fmt)


def _n(name, rows, h, x, fmt, post, gate):
    """r' = r + scale * gate * norm(f), then norm(r') in 4 bits."""
    return dict(name=name, op="norm", rows=rows, h=h, x=x, fmt=fmt, post=post, gate=gate)


def listed():
    return [
        # activations of sixteen sequences that decode one token each
        _q("quantize 16x4096", 16, 4096, "bf16", NV, g=0.5),
        # a prompt's activations before a down projection
        _q("quantize 4096x14336", 4096, 14336, "bf16", NV),
        # routed token rows, sorted by expert, out of a wider buffer
        _q("quantize experts 1999x4112", 1999, 4112, "f16", MX, experts=8, pad=48),
        # one token through a down projection: the weights are the work
        _p("product 1x4096x14336", 1, 4096, 14336, "bf16", NV),
        # a batch of 64 decoding sequences through an up projection
        _p("product 64x11008x4096", 64, 11008, 4096, "bf16", MX, act="gelu"),
        # sizes that fit no tile, fp32 result added to what is there
        _p("product 333x1002x2080", 333, 1002, 2080, "f32", NV, beta=1.0),
        # the square product that dense throughput is quoted on
        _p("product 4096x4096x4096", 4096, 4096, 4096, "bf16", NV),
        # a prompt through an up projection
        _p("product 4096x14336x4096", 4096, 14336, 4096, "f16", MX),
        # sixteen decoding tokens, each routed to two of eight experts
        _g("grouped 32x8x14336x4096", 32, 8, 14336, 4096, "bf16", NV),
        # a prompt of 4096 routed rows, popular experts first
        _g("grouped 4096x8x14336x4096", 4096, 8, 14336, 4096, "bf16", NV),
        # one token between two layers
        _n("norm 1x4096", 1, 4096, "bf16", NV, True, ""),
        # a prompt between two layers: post-norm, one gate per channel
        _n("norm 4096x4096", 4096, 4096, "bf16", NV, True, "channel"),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(max(v, lo), hi)
    return v + 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "grouped", "norm"])
    fmt = rng.choice([NV, MX])
    x = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "quantize":
        c = _q("", _log(rng, 1, 4096), _log(rng, 64, 14336), x, fmt, rng.choice([0, 0, 8, 64]), rng.choice([0, 0, 8, 3]),
               0.5 if fmt == NV and rng.random() < 0.5 else 1.0)
    elif op == "product":
        # the row stride of packed codes is a multiple of 32 values; K is not
        c = _p("", _log(rng, 1, 4096), _log(rng, 64, 14336), _log(rng, 64, 4096), x, fmt,
               rng.choice(["", "", "gelu", "relu"]), rng.choice([0.0, 0.0, 0.5]))
    elif op == "grouped":
        c = _g("", _log(rng, 4, 4096), rng.choice([2, 8, 8, 32]), _log(rng, 64, 4096), _log(rng, 64, 4096), x, fmt)
    else:
        c = _n("", _log(rng, 1, 4096), _log(rng, 64, 14336), x, fmt, rng.random() < 0.5,
               rng.choice(["", "channel", "element"]))
    del c["name"]
    return c


# ---- the formats, in elementary operations ----------------------------------

def _ceil(a, b):
    return -(-a // b)


def _blocks(x, b):
    """[rows, k] -> [rows, blocks, b] in fp32, the last block padded with zeros."""
    rows, k = x.shape
    n = _ceil(k, b)
    if n * b == k:
        return x.float().view(rows, n, b)
    y = torch.zeros(rows, n * b, dtype=torch.float32, device=x.device)
    y[:, :k] = x
    return y.view(rows, n, b)


def _quantize(x, fmt, g=1.0):
    """Codes 0..15 [rows, k] (uint8) and scale bytes [rows, blocks] (uint8)."""
    rows, k = x.shape
    v = _blocks(x, BLOCK[fmt])
    amax = v.abs().amax(-1)
    fine = amax <= torch.finfo(torch.float32).max
    if fmt == NV:
        # a tensor divides; a Python number would be turned into a factor
        top = torch.full((1,), 6.0 * g, dtype=torch.float32, device=x.device)
        s8 = torch.clamp(torch.where(fine, amax, 0.0) / top, max=448.0).to(torch.float8_e4m3fn)
        s = s8.float() * g
        byte = torch.where(fine, s8.view(torch.uint8), 0x7F)
    else:
        # floor(log2 amax) is the exponent field; E8M0 byte e stands for 2^(e - 127)
        e = (amax.view(torch.int32) >> 23) - 2
        e = torch.clamp(e, min=0)
        # 2^(e - 127): the exponent field, and the one subnormal value for e = 0
        s = torch.where(e > 0, e << 23, 1 << 22).view(torch.float32)
        byte = torch.where(fine, e, 255).to(torch.uint8)
    live = ((s > 0) & fine).unsqueeze(-1)
    w = torch.where(live, v / s.unsqueeze(-1), 0.0)
    a = w.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + torch.signbit(w).to(torch.uint8) * 8
    return code.view(rows, -1)[:, :k], byte


def _pack(code):
    """Codes [rows, k] -> bytes [rows, ld / 2], ld = k rounded up to 32."""
    rows, k = code.shape
    full = torch.zeros(rows, _ceil(k, 32) * 32, dtype=torch.uint8, device=code.device)
    full[:, :k] = code
    return full[:, 0::2] | (full[:, 1::2] << 4)


def _unpack(packed, k):
    return torch.stack([packed & 15, packed >> 4], -1).view(packed.shape[0], -1)[:, :k]


def _tile(byte, at=None, tiles=None):
    """Scale bytes [rows, blocks] -> the stored layout.  `at`: the padded row
    of each row (rows sorted by expert), `tiles` atom rows in all."""
    rows, n = byte.shape
    tiles = _ceil(rows, 128) if tiles is None else tiles
    atoms = _ceil(n, 4)
    full = torch.zeros(tiles * 128, atoms * 4, dtype=torch.uint8, device=byte.device)
    if at is None:
        full[:rows, :n] = byte
    else:
        full[at, :n] = byte
    return full.view(tiles, 4, 32, atoms, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untile(flat, tiles, n):
    """The stored layout -> scale bytes [tiles * 128, n]."""
    atoms = _ceil(n, 4)
    return flat.view(tiles, atoms, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(tiles * 128, atoms * 4)[:, :n]


def _scale_values(byte, fmt):
    return byte.view(SCALE_TYPE[fmt]).float()


def _value_table(device):
    t = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(t + [-v for v in t], dtype=torch.float32, device=device)


def _dequantize(packed, byte, k, fmt):
    """fp32 values [rows, k] of packed codes and untiled scale bytes."""
    v = _value_table(packed.device)[_unpack(packed, k).int()]
    return v * _scale_values(byte, fmt).repeat_interleave(BLOCK[fmt], 1)[:, :k]


def _expert_rows(offsets, rows):
    """Padded scale row of every token row: experts start on atom rows."""
    sizes = offsets[1:] - offsets[:-1]
    tiles = (sizes + 127) // 128
    start = (torch.cumsum(tiles, 0) - tiles) * 128
    r = torch.arange(rows, device=offsets.device)
    e = torch.searchsorted(offsets[1:].contiguous(), r, right=True)
    return start[e] + r - offsets[e]


def _expert_tiles(rows, experts):
    return rows // 128 + experts


# ---- inputs -----------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _activations(gen, rows, k):
    """Normal values with a few loud channels, as hidden states have them."""
    loud = torch.where(torch.rand(k, generator=gen, device="cuda") < 0.01, 12.0, 1.0)
    return _normal(gen, rows, k) * loud


def _offsets(gen, rows, experts):
    """Row offsets of experts whose popularity falls off as 1 / rank^1.2."""
    p = torch.arange(1, experts + 1, device="cuda", dtype=torch.float64) ** -1.2
    p = p[torch.randperm(experts, generator=gen, device="cuda")]
    pick = torch.multinomial(p, rows, replacement=True, generator=gen)
    count = torch.bincount(pick, minlength=experts)
    return torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(count, 0)]).int()


def _weights(gen, n, k, fmt):
    code, byte = _quantize(_normal(gen, n, k) * 0.02, fmt)
    return _pack(code), _tile(byte)


def prepare(case, seed):
    gen, s = _gen(seed), dict(case)
    fmt = case["fmt"]
    if case["op"] == "quantize":
        rows, k, experts = case["rows"], case["k"], case["experts"]
        wide = _activations(gen, rows, k + case["pad"]).to(TYPES[case["x"]])
        s["x_values"] = wide[:, :k]
        s["offsets"] = _offsets(gen, rows, experts) if experts else None
        tiles = _expert_tiles(rows, experts) if experts else _ceil(rows, 128)
        s["packed"] = torch.zeros(rows, _ceil(k, 32) * 16, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.zeros(tiles * 512 * _ceil(k, 4 * BLOCK[fmt]), dtype=torch.uint8, device="cuda")
        s["codes"] = torch.empty(rows, k, dtype=torch.float8_e4m3fn, device="cuda")
    elif case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        code, byte = _quantize(_activations(gen, m, k), fmt)
        s["a"], s["sa"] = _pack(code), _tile(byte)
        s["b"], s["sb"] = _weights(gen, n, k, fmt)
        s["alpha"] = 1.5
        s["c"] = _normal(gen, m, n).to(TYPES[case["d"]]) if case["beta"] else None
        s["bias"] = _normal(gen, n).to(torch.bfloat16) if case["act"] else None
        s["out"] = torch.empty(m, n, dtype=TYPES[case["d"]], device="cuda")
    elif case["op"] == "grouped":
        rows, experts, n, k = case["rows"], case["experts"], case["n"], case["k"]
        s["offsets"] = _offsets(gen, rows, experts)
        s["host_offsets"] = s["offsets"].tolist()  # the plain form cuts its products on the host
        code, byte = _quantize(_activations(gen, rows, k), fmt)
        s["a"] = _pack(code)
        s["sa"] = _tile(byte, _expert_rows(s["offsets"], rows), _expert_tiles(rows, experts))
        w = [_weights(gen, n, k, fmt) for _ in range(experts)]
        s["b"], s["sb"] = torch.stack([v[0] for v in w]), torch.stack([v[1] for v in w])
        s["expert_alpha"] = torch.rand(experts, generator=gen, device="cuda") + 0.5
        s["out"] = torch.empty(rows, n, dtype=TYPES[case["d"]], device="cuda")
    else:
        rows, h, x = case["rows"], case["h"], TYPES[case["x"]]
        s["f"] = _activations(gen, rows, h).to(x)
        s["r"] = (3.0 * _normal(gen, rows, h)).to(x)
        s["pre"] = (1.0 + 0.1 * _normal(gen, h)).to(x)
        s["post_w"] = (0.3 + 0.1 * _normal(gen, h)).to(x) if case["post"] else None
        s["g_values"] = None
        if case["gate"]:
            s["g_values"] = torch.tanh(_normal(gen, *((h,) if case["gate"] == "channel" else (rows, h)))).to(x)
        s["eps"], s["res_scale"] = 1e-5, 0.7
        s["new_r"] = torch.empty(rows, h, dtype=x, device="cuda")
        s["packed"] = torch.zeros(rows, _ceil(h, 32) * 16, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.zeros(_ceil(rows, 128) * 512 * _ceil(h, 4 * BLOCK[fmt]), dtype=torch.uint8, device="cuda")
        s["codes"] = torch.empty(rows, h, dtype=torch.float8_e4m3fn, device="cuda")
    return s


# ---- one pass ---------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _finish(acc, s):
    """alpha, C, bias and activation in fp32, one rounding."""
    y = s["alpha"] * acc
    if s["c"] is not None:
        y = y + s["beta"] * s["c"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if s["act"] == "relu":
        y = torch.where(y < 0, 0.0, y)
    if s["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * 0.7071067811865476))
    return y.to(TYPES[s["d"]])


def _run_plain(s):
    fmt, op = s["fmt"], s["op"]
    blk = BLOCK[fmt]
    if op == "quantize":
        rows, k = s["rows"], s["k"]
        code, byte = _quantize(s["x_values"], fmt, s["g"])
        if s["experts"]:
            stored = _tile(byte, _expert_rows(s["offsets"], rows), _expert_tiles(rows, s["experts"]))
        else:
            stored = _tile(byte)
        return {"codes": _value_table(code.device)[code.int()].to(torch.float8_e4m3fn), "scales": stored.view(SCALE_TYPE[fmt])}
    if op == "product":
        m, n, k = s["m"], s["n"], s["k"]
        nb = _ceil(k, blk)
        a = _dequantize(s["a"], _untile(s["sa"], _ceil(m, 128), nb)[:m], k, fmt)
        b = _dequantize(s["b"], _untile(s["sb"], _ceil(n, 128), nb)[:n], k, fmt)
        return _finish(a @ b.t(), s)
    if op == "grouped":
        rows, n, k, off = s["rows"], s["n"], s["k"], s["host_offsets"]
        nb = _ceil(k, blk)
        sa = _untile(s["sa"], _expert_tiles(rows, s["experts"]), nb)[_expert_rows(s["offsets"], rows)]
        a = _dequantize(s["a"], sa, k, fmt)
        y = torch.empty(rows, n, dtype=torch.float32, device=a.device)
        # one product per expert that has rows: cutting here is cheaper than
        # padding every expert to the most popular one's rows
        for e in range(s["experts"]):
            if off[e + 1] > off[e]:
                b = _dequantize(s["b"][e], _untile(s["sb"][e], _ceil(n, 128), nb)[:n], k, fmt)
                torch.matmul(a[off[e]:off[e + 1]], b.t(), out=y[off[e]:off[e + 1]])
                y[off[e]:off[e + 1]] *= s["expert_alpha"][e]
        return y.to(TYPES[s["d"]])
    u = s["f"].float()
    if s["post_w"] is not None:
        u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + s["eps"]) * s["post_w"].float()
    if s["g_values"] is not None:
        u = u * s["g_values"].float()
    new_r = (s["r"].float() + s["res_scale"] * u).to(TYPES[s["x"]])
    v = new_r.float()
    y = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + s["eps"]) * s["pre"].float()
    code, byte = _quantize(y, fmt)
    return {"residual": new_r, "codes": _value_table(code.device)[code.int()].to(torch.float8_e4m3fn),
            "scales": _tile(byte).view(SCALE_TYPE[fmt])}


_handle = None


def _plan(qg, s):
    """The descriptors that a program keeps beside its buffers."""
    global _handle
    if _handle is None:
        _handle = qg.gemm_create()
    h, op = _handle, s["op"]
    fmt = {NV: qg.GEMM_NVFP4, MX: qg.GEMM_MXFP4}[s["fmt"]]
    four = lambda t, k: qg.mx_layout(t, k)  # noqa: E731
    if op == "quantize":
        q = four(s["packed"], s["k"])
        exp = (qg.ptr(s["offsets"]), s["experts"])
        sc = (qg.ptr(s["scales"]), s["scales"].numel())
        return [
            (qg.gemm_mx_quantize, (h, fmt, s["g"], qg.ptr(s["x_values"]), qg.row_major(s["x_values"]), qg.ptr(s["packed"]), q, *sc, *exp)),
            (qg.gemm_mx_dequantize, (h, fmt, 1.0, qg.ptr(s["packed"]), q, *sc, qg.ptr(s["codes"]), qg.row_major(s["codes"]), *exp)),
        ]
    if op == "product":
        o = qg.gemm_op_t()
        if s["bias"] is not None:
            o.epilogue = qg.GEMM_EPILOGUE_BIAS | {"gelu": qg.GEMM_EPILOGUE_GELU, "relu": qg.GEMM_EPILOGUE_RELU}[s["act"]]
            o.bias, o.bias_type = qg.ptr(s["bias"]), qg.GEMM_BF16
        c = s["c"]
        return [(qg.gemm_run_mx, (h, o, fmt, s["alpha"], qg.ptr(s["a"]), four(s["a"], s["k"]), qg.ptr(s["sa"]), s["sa"].numel(),
                                  qg.ptr(s["b"]), qg.mx_layout_b(s["b"], s["k"]), qg.ptr(s["sb"]), s["sb"].numel(), s["beta"],
                                  qg.ptr(c), None if c is None else qg.row_major(c), qg.ptr(s["out"]), qg.row_major(s["out"])))]
    if op == "grouped":
        return [(qg.gemm_run_mx_grouped, (h, qg.gemm_op_t(), fmt, 1.0, qg.ptr(s["expert_alpha"]), qg.ptr(s["a"]), four(s["a"], s["k"]),
                                          qg.ptr(s["sa"]), s["sa"].numel(), qg.ptr(s["b"]), qg.mx_layout_b(s["b"], s["k"]), qg.ptr(s["sb"]),
                                          s["sb"].numel(), 0.0, None, None, qg.ptr(s["out"]), qg.row_major(s["out"]),
                                          qg.ptr(s["offsets"]), s["experts"]))]
    n = qg.gemm_mx_norm_t(format=fmt, tensor_scale=1.0, eps=s["eps"], residual_scale=s["res_scale"])
    n.pre_weight, n.weight_type = qg.ptr(s["pre"]), qg.row_major(s["r"]).type
    if s["post_w"] is not None:
        n.post_weight = qg.ptr(s["post_w"])
    if s["g_values"] is not None:
        n.gate, n.gate_type, n.gate_ld = qg.ptr(s["g_values"]), n.weight_type, s["h"] if s["gate"] == "element" else 0
    q, sc = four(s["packed"], s["h"]), (qg.ptr(s["scales"]), s["scales"].numel())
    return [
        (qg.gemm_mx_norm_quantize, (h, n, qg.ptr(s["f"]), qg.row_major(s["f"]), qg.ptr(s["r"]), qg.row_major(s["r"]),
                                    qg.ptr(s["new_r"]), qg.row_major(s["new_r"]), qg.ptr(s["packed"]), q, *sc)),
        (qg.gemm_mx_dequantize, (h, fmt, 1.0, qg.ptr(s["packed"]), q, *sc, qg.ptr(s["codes"]), qg.row_major(s["codes"]), None, 0)),
    ]


def _run_own(s):
    import quantized_gemm_tcgen05_gb300 as qg

    if "plan" not in s:
        s["plan"] = _plan(qg, s)
    stream = qg.current_stream()
    for call, args in s["plan"]:
        rc = call(*args, stream)
        if rc:
            raise qg.GemmError(rc, call.__name__)
    if s["op"] in ("product", "grouped"):
        return s["out"]
    out = {"codes": s["codes"], "scales": s["scales"].view(SCALE_TYPE[s["fmt"]])}
    if s["op"] == "norm":
        out["residual"] = s["new_r"]
    return out


# ---- what a pass cannot do without ------------------------------------------

def _bits(fmt, rows, k):
    """Bytes of rows x k packed values and their scales, without padding."""
    return rows * (_ceil(k, 2) + _ceil(k, BLOCK[fmt]))


def work(case):
    size, fmt = {"f32": 4, "f16": 2, "bf16": 2}, case["fmt"]
    if case["op"] == "quantize":
        rows, k = case["rows"], case["k"]
        # values in; codes and scales out; the codes once more as 8-bit floats
        return {"bytes": rows * k * (size[case["x"]] + 1) + 2 * _bits(fmt, rows, k), "flops": 3 * rows * k}
    if case["op"] == "product":
        m, n, k, d = case["m"], case["n"], case["k"], size[case["d"]]
        return {"bytes": _bits(fmt, m, k) + _bits(fmt, n, k) + m * n * d * (2 if case["beta"] else 1), "flops": 2 * m * n * k}
    if case["op"] == "grouped":
        rows, n, k = case["rows"], case["n"], case["k"]
        # the experts that 1 / rank^1.2 popularity is expected to give rows
        p = [i ** -1.2 for i in range(1, case["experts"] + 1)]
        met = sum(1.0 - (1.0 - v / sum(p)) ** rows for v in p)
        return {"bytes": _bits(fmt, rows, k) + met * _bits(fmt, n, k) + rows * n * size[case["d"]], "flops": 2 * rows * n * k}
    rows, h, x = case["rows"], case["h"], size[case["x"]]
    gate = {"": 0, "channel": h, "element": rows * h}[case["gate"]]
    return {"bytes": rows * h * (3 * x + 1) + 2 * _bits(fmt, rows, h) + x * (gate + h * (2 if case["post"] else 1)),
            "flops": 12 * rows * h}


# ---- the definitions in 64 bits ---------------------------------------------

def _pow2(e):
    """2^e exactly: the exponent field of a double."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _floor_log2(v):
    return torch.frexp(v)[1] - 1


def _exact_e2m1(packed, k):
    """Values by the format's definition: sign, 2-bit exponent, 1-bit mantissa."""
    q = torch.empty(packed.shape[0], packed.shape[1] * 2, dtype=torch.int32, device=packed.device)
    q[:, 0::2] = packed.int() % 16
    q[:, 1::2] = packed.int() // 16
    q = q[:, :k]
    e, m = (q // 2) % 4, (q % 2).double()
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * _pow2(e - 1))
    return torch.where(q >= 8, -mag, mag)


def _exact_scale(flat, row, nb, fmt):
    """Scale values [rows, nb] read out of the stored layout by its formula."""
    j = torch.arange(nb, device=flat.device)
    atoms = _ceil(nb, 4)
    at = (row[:, None] // 128 * atoms + j // 4) * 512 + row[:, None] % 32 * 16 + row[:, None] % 128 // 32 * 4 + j % 4
    b = flat[at.long()].int()
    if fmt == MX:
        return _pow2(b - 127)
    e, m = b // 8, (b % 8).double()
    return torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * _pow2(e - 7))


def _exact_values(packed, flat, row, k, fmt):
    nb = _ceil(k, BLOCK[fmt])
    block = torch.arange(k, device=packed.device) // BLOCK[fmt]
    return _exact_e2m1(packed, k) * _exact_scale(flat, row, nb, fmt)[:, block]


def _exact_quantize(x, fmt, g):
    """Codes' values and scales' values of x (fp64), by the definition."""
    rows, k = x.shape
    b = BLOCK[fmt]
    v = torch.nn.functional.pad(x, (0, -k % b)).view(rows, -1, b)
    amax = v.abs().amax(-1)
    if fmt == NV:
        t = torch.clamp(amax / torch.full_like(amax, 6 * g), max=448.0)  # a true division, as above
        step = _pow2(torch.clamp(_floor_log2(t), min=-6) - 3)
        s = torch.round(t / step) * step
        u = s * g
    else:
        s = u = _pow2(torch.where(amax > 0, torch.clamp(_floor_log2(amax) - 2, min=-127), -127))
    w = torch.where(u[..., None] > 0, v / torch.where(u > 0, u, 1.0)[..., None], 0.0)
    step = _pow2(torch.clamp(_floor_log2(w.abs()), 0, 2) - 1)
    return (torch.round(w / step) * step).clamp(-6.0, 6.0).view(rows, -1)[:, :k], s


def exact(case, seed):
    s = prepare(case, seed)
    fmt, op = case["fmt"], case["op"]
    if op == "quantize":
        codes, scale = _exact_quantize(s["x_values"].double(), fmt, case["g"])
        rows, nb = scale.shape
        row = torch.arange(rows, device="cuda")
        if case["experts"]:
            off = s["offsets"].tolist()
            start, at = 0, []
            for e in range(case["experts"]):
                at.append(start + torch.arange(off[e + 1] - off[e], device="cuda"))
                start += _ceil(off[e + 1] - off[e], 128) * 128
            row = torch.cat(at)
        atoms = _ceil(nb, 4)
        # a padded byte is zero: E4M3 0, E8M0 2^-127
        flat = torch.full((s["scales"].numel(),), 0.0 if fmt == NV else 2.0 ** -127, dtype=torch.float64, device="cuda")
        j = torch.arange(nb, device="cuda")
        flat[(row[:, None] // 128 * atoms + j // 4) * 512 + row[:, None] % 32 * 16 + row[:, None] % 128 // 32 * 4 + j % 4] = scale
        return {"codes": codes, "scales": flat}
    if op == "product":
        a = _exact_values(s["a"], s["sa"], torch.arange(case["m"], device="cuda"), case["k"], fmt)
        b = _exact_values(s["b"], s["sb"], torch.arange(case["n"], device="cuda"), case["k"], fmt)
        y = s["alpha"] * (a @ b.t())
        if case["beta"]:
            y += case["beta"] * s["c"].double()
        if case["act"]:
            y += s["bias"].double()
            y = torch.clamp(y, min=0.0) if case["act"] == "relu" else y * (1 + torch.erf(y / math.sqrt(2.0))) / 2
        return y
    if op == "grouped":
        off, start, parts = s["offsets"].tolist(), 0, []
        for e in range(case["experts"]):
            m = off[e + 1] - off[e]
            if m:
                a = _exact_values(s["a"][off[e]:off[e + 1]], s["sa"], start + torch.arange(m, device="cuda"), case["k"], fmt)
                b = _exact_values(s["b"][e], s["sb"][e], torch.arange(case["n"], device="cuda"), case["k"], fmt)
                parts.append(s["expert_alpha"][e].double() * (a @ b.t()))
            start += _ceil(m, 128) * 128
        return torch.cat(parts)
    f, r = s["f"].double(), s["r"].double()
    if s["post_w"] is not None:
        f = f / torch.sqrt(f.square().mean(-1, keepdim=True) + s["eps"]) * s["post_w"].double()
    if s["g_values"] is not None:
        f = f * s["g_values"].double()
    # the codes are decided by roundings of values that fp32 does not hold
    # exactly: they have no one value in 64 bits
    return {"residual": r + s["res_scale"] * f, "codes": None, "scales": None}
