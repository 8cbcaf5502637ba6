"""The example block (examples/mx_block.py) end to end: every product against
numpy in 64 bits on the operands that the step really used, and the residual
from the block's real output."""
import os
import sys

import numpy as np
import pytest
import torch

import mx_ref as R
import oracle
import quantized_gemm_tcgen05_gb300 as qg
import synth

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import mx_block  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h():
    h = qg.gemm_create()
    yield h
    qg.gemm_destroy(h)


def f64(t):
    return t.double().cpu().numpy()


def operand(o, fmt, rows=None):
    """Values of an MxOperand; rows: scale row of every row."""
    code = R.unpack(o.codes.cpu().numpy(), o.k)
    nb = R.ceil(o.k, R.BLOCK[fmt])
    if code.ndim == 3:
        per = o.scales.numel() // code.shape[0]
        flat = o.scales.cpu().numpy().reshape(code.shape[0], per)
        at = R.scale_at(np.arange(o.rows)[:, None], np.arange(nb)[None], R.ceil(nb, 4))
        return np.stack([R.dequantize(code[e], flat[e][at], fmt) for e in range(code.shape[0])])
    rows = np.arange(o.rows) if rows is None else rows
    at = R.scale_at(rows[:, None], np.arange(nb)[None], R.ceil(nb, 4))
    return R.dequantize(code, o.scales.cpu().numpy()[at], fmt)


def close(got, ref, bound):
    tol = 1e-5 * bound + 1e-6 + oracle.ulp(synth.BF16, ref)
    assert (np.abs(f64(got) - ref) <= tol).all()


@pytest.mark.parametrize("fmt", [qg.GEMM_NVFP4, qg.GEMM_MXFP4])
@pytest.mark.parametrize("tokens,counts", [(1, None), (37, None), (300, None), (40, [7, 0, 30, 3]), (1, [0, 1]), (300, [0, 170, 130])])
def test_block(h, fmt, tokens, counts):
    hidden, inner = 320, 704
    E = len(counts) if counts else 0
    w = mx_block.Weights(h, hidden, inner, E, fmt, seed=tokens)
    off = np.concatenate([[0], np.cumsum(counts)]) if E else np.array([0, tokens])
    offd = torch.from_numpy(off.astype(np.int32)).cuda() if E else None
    b = mx_block.Block(h, w, tokens, offd)
    x = torch.randn(tokens, hidden, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    new = b.step(x)
    assert qg.gemm_device_status(h, qg.current_stream()) == 0
    rows = R.expert_rows(off) if E else None
    a, q = operand(b.normed, fmt, rows), operand(b.inner_q, fmt, rows)
    up, down = operand(w.up, fmt), operand(w.down, fmt)
    if not E:
        up, down = up[None], down[None]
    f32 = np.float32
    for e in range(max(E, 1)):
        s = slice(off[e], off[e + 1])
        us, ds = float(f32(w.up_scale)), float(f32(w.down_scale))
        bias = f64(w.up_bias)
        y = us * a[s] @ up[e].T + bias
        ref = (0.5 * torch.from_numpy(y) * (1 + torch.erf(torch.from_numpy(y) / 2 ** 0.5))).numpy()
        close(b.inner[s], ref, 1.129 * (us * np.abs(a[s]) @ np.abs(up[e]).T + np.abs(bias)))
        close(b.out[s], ds * q[s] @ down[e].T, ds * np.abs(q[s]) @ np.abs(down[e]).T)
    f = f64(b.out)
    u = f / np.sqrt((f * f).mean(-1, keepdims=True) + 1e-5) * f64(w.norm_after) * f64(w.gate)
    want = f64(x) + u
    assert (np.abs(f64(new) - want) <= 4e-6 * np.abs(u) + 2.0 ** -22 * np.abs(want) + oracle.ulp(synth.BF16, want)).all()
    # the whole block is what its unquantised form gives, to 4 bits' accuracy
    assert torch.isfinite(new.float()).all()
