"""Plain definitions, in 64 bits or in the stated fp32 steps, of the operators of
include/gemm_moe.h and include/gemm_s8.h, for the tests."""
import numpy as np
import torch

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = {torch.float32: 2.0 ** -23, torch.float16: 2.0 ** -10, torch.bfloat16: 2.0 ** -7}


def route(logits, topk, score="softmax", bias=None, groups=1, group_topk=1, group_best=1, renormalize=True, scale=1.0):
    """ids, weights, rows, offsets of logits [tokens, experts] (fp64), token by token."""
    tokens, experts = logits.shape
    ids = np.full((tokens, topk), -1, dtype=np.int32)
    w = np.zeros((tokens, topk))
    for t in range(tokens):
        l = logits[t].astype(np.float64)
        if np.isnan(l).any() or (score == "softmax" and np.isposinf(l).any()) or (bias is not None and np.isnan(bias).any()):
            w[t] = np.nan
            continue
        live = l > -np.inf
        if not live.any():
            continue
        with np.errstate(over="ignore"):
            if score == "softmax":
                e = np.where(live, np.exp(l - l.max()), 0.0)
                s = e / e.sum()
            else:
                s = 1.0 / (1.0 + np.exp(-l))
        b = np.zeros(experts) if bias is None else bias.astype(np.float64)
        live &= b > -np.inf
        c = np.where(live, s + b, -np.inf)
        if groups > 1:
            size = experts // groups
            total = []
            for g in range(groups):
                have = sorted((c[e] for e in range(g * size, (g + 1) * size) if live[e]), reverse=True)[:group_best]
                total.append(sum(have) if have else -np.inf)
            kept = sorted(range(groups), key=lambda g: (-total[g], g))[:group_topk]
            live &= np.isin(np.arange(experts) // size, kept)
        key = l if bias is None else c
        order = sorted((e for e in range(experts) if live[e]), key=lambda e: (-key[e], e))[:topk]
        ids[t, :len(order)] = order
        if order:
            if renormalize:
                # of the logarithms, so that nothing underflows
                x = l[order]
                q = -np.logaddexp(0.0, -x) if score == "sigmoid" else x
                v = np.exp(q - q.max())
                v = v / v.sum()
            else:
                v = s[order]
            w[t, :len(order)] = v * scale
    rows = np.full(tokens * topk, -1, dtype=np.int32)
    flat = ids.reshape(-1)
    offsets, at = [0], 0
    for e in range(experts):
        mine = np.nonzero(flat == e)[0]
        rows[mine] = at + np.arange(len(mine))
        at += len(mine)
        offsets.append(at)
    return ids, w, rows.reshape(tokens, topk), np.array(offsets, dtype=np.int32)


def quantize(x):
    """int8 codes and fp32 scales of x [rows, cols], every step rounded to fp32."""
    x = x.float().cpu().numpy()
    q = np.zeros(x.shape, dtype=np.int8)
    s = np.zeros(x.shape[0], dtype=np.float32)
    for r in range(x.shape[0]):
        if not np.isfinite(x[r]).all():
            s[r] = np.nan
            continue
        amax = np.float32(np.abs(x[r]).max(initial=0.0))
        scale = np.float32(amax / np.float32(127.0))
        tiny = scale < np.float32(2.0 ** -126)
        f = np.float32(2.0 ** 126) if tiny else np.float32(np.float32(127.0) / amax)
        s[r] = np.float32(2.0 ** -126) if tiny else scale
        q[r] = np.rint((x[r] * f).astype(np.float32)).astype(np.int8)
    return q, s


def sums(a, b):
    """Exact integer sums a b^T of int8 matrices (fp64 holds them below 2^53)."""
    return (a.double().cpu() @ b.double().cpu().t()).numpy().astype(np.int64)


def product(total, alpha, sa, sb, d, beta=0.0, c=None, bias=None, relu=False):
    """The stated fp32 steps after an exact sum, rounded to torch type d."""
    f = np.float32
    token = np.full(total.shape[0], f(alpha)) if sa is None else (f(alpha) * sa.cpu().numpy()).astype(f)
    channel = np.ones(total.shape[1], dtype=f) if sb is None else sb.cpu().numpy()
    with np.errstate(over="ignore", invalid="ignore"):
        v = (total.astype(f) * token[:, None]).astype(f)
        v = (v * channel[None, :]).astype(f)
        if beta != 0.0:
            v = (v + (f(beta) * c.float().cpu().numpy()).astype(f)).astype(f)
        if bias is not None:
            v = (v + bias.float().cpu().numpy()[None, :]).astype(f)
        if relu:
            v = np.where(v < 0, f(0), v)
    return torch.from_numpy(v).to(d)
