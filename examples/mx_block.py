"""A transformer block's feed-forward half in 4 bits, dense or with experts, for a
prompt or for single tokens, out of the library's microscaled operators:

    norm before the block, quantising      gemm_mx_norm_quantize
    up product + bias + GELU               gemm_run_mx / gemm_run_mx_grouped
    quantise                               gemm_mx_quantize
    down product                           gemm_run_mx / gemm_run_mx_grouped
    norm after the block, gate, residual,
    norm before the next one, quantising   gemm_mx_norm_quantize

Weights are quantised once.  Run it for a time per step:

    python examples/mx_block.py --tokens 16 --hidden 4096 --inner 14336 --experts 8
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_gemm_tcgen05_gb300 as qg  # noqa: E402


def check(rc, what):
    if rc:
        raise qg.GemmError(rc, what)


class Weights:
    """The block's weights: matrices in 4 bits with one fp32 scale each."""

    def __init__(self, h, hidden, inner, experts=0, fmt=qg.GEMM_NVFP4, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        num = max(experts, 1)
        new = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
        self.hidden, self.inner, self.experts, self.fmt = hidden, inner, experts, fmt
        self.up, self.up_scale = self._quantize(h, new(num, inner, hidden) * hidden ** -0.5)
        self.down, self.down_scale = self._quantize(h, new(num, hidden, inner) * inner ** -0.5)
        self.up_bias = (0.1 * new(inner)).bfloat16()
        self.norm_before = (1 + 0.1 * new(hidden)).bfloat16()
        self.norm_after = (1 + 0.1 * new(hidden)).bfloat16()
        self.norm_next = (1 + 0.1 * new(hidden)).bfloat16()
        self.gate = torch.tanh(new(hidden)).bfloat16()
        if experts:
            # one scale per expert: a factor on alpha, expert by expert
            self.up_alpha = torch.full((experts,), self.up_scale, device="cuda")
            self.down_alpha = torch.full((experts,), self.down_scale, device="cuda")

    def _quantize(self, h, w):
        # NVFP4: the tensor scale that puts the largest block scale at E4M3's top
        scale = float(w.abs().max()) / (6 * 448) if self.fmt == qg.GEMM_NVFP4 else 1.0
        w = w.bfloat16()
        if not self.experts:
            w = w[0]
        o = qg.MxOperand(self.fmt, w.shape[-2], w.shape[-1], num=max(self.experts, 1) if w.dim() == 3 else 1)
        codes, layout, scales, size = o.args()
        check(qg.gemm_mx_quantize(h, self.fmt, scale, qg.ptr(w), qg.row_major(w), codes, layout, scales, size, None, 0,
                                  qg.current_stream()), "gemm_mx_quantize")
        return o, scale


class Block:
    """Buffers for `tokens` rows and the step itself.  With experts, `offsets`
    (device int32[experts + 1]) says which of the rows, sorted by expert, are
    whose; the residual stream then is in that order too."""

    def __init__(self, h, weights, tokens, offsets=None):
        w = self.w = weights
        self.h, self.tokens, self.offsets = h, tokens, offsets
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.normed = qg.MxOperand(w.fmt, tokens, w.hidden, num_experts=w.experts)
        self.inner = torch.empty(tokens, w.inner, **bf)
        self.inner_q = qg.MxOperand(w.fmt, tokens, w.inner, num_experts=w.experts)
        self.out = torch.empty(tokens, w.hidden, **bf)
        self.x = torch.empty(tokens, w.hidden, **bf)
        self.next = qg.MxOperand(w.fmt, tokens, w.hidden)

    def _norm(self, f, r, out, pre, to, by_expert=False):
        w, n = self.w, qg.gemm_mx_norm_t(format=self.w.fmt, tensor_scale=1.0, eps=1e-5, residual_scale=1.0)
        n.weight_type = n.gate_type = qg.GEMM_BF16
        n.pre_weight = qg.ptr(pre)
        if by_expert:
            n.expert_offsets, n.num_experts = qg.ptr(self.offsets), w.experts
        if f is not None:
            n.post_weight, n.gate = qg.ptr(w.norm_after), qg.ptr(w.gate)
        lay = lambda t: None if t is None else qg.row_major(t)  # noqa: E731
        check(qg.gemm_mx_norm_quantize(self.h, n, qg.ptr(f), lay(f), qg.ptr(r), lay(r), qg.ptr(out), lay(out), *to.args(),
                                       qg.current_stream()), "gemm_mx_norm_quantize")

    def _product(self, a, b, alpha, expert_alpha, op, out):
        args = (*a.args(), *b.args(b=True), 0.0, None, None, qg.ptr(out), qg.row_major(out))
        if self.w.experts:
            check(qg.gemm_run_mx_grouped(self.h, op, self.w.fmt, 1.0, qg.ptr(expert_alpha), *args, qg.ptr(self.offsets),
                                         self.w.experts, qg.current_stream()), "gemm_run_mx_grouped")
        else:
            check(qg.gemm_run_mx(self.h, op, self.w.fmt, alpha, *args, qg.current_stream()), "gemm_run_mx")

    def step(self, x):
        """x: [tokens, hidden] bf16 residual stream.  Returns the new residual
        stream; `self.next` holds the next block's operand."""
        w = self.w
        off, E = qg.ptr(self.offsets), w.experts
        self._norm(None, x, None, w.norm_before, self.normed, by_expert=E > 0)
        up = qg.gemm_op_t(epilogue=qg.GEMM_EPILOGUE_BIAS | qg.GEMM_EPILOGUE_GELU, bias=qg.ptr(w.up_bias),
                          bias_type=qg.GEMM_BF16)
        self._product(self.normed, w.up, w.up_scale, w.up_alpha if E else None, up, self.inner)
        check(qg.gemm_mx_quantize(self.h, w.fmt, 1.0, qg.ptr(self.inner), qg.row_major(self.inner), *self.inner_q.args(),
                                  off, E, qg.current_stream()), "gemm_mx_quantize")
        self._product(self.inner_q, w.down, w.down_scale, w.down_alpha if E else None, qg.gemm_op_t(), self.out)
        self._norm(self.out, x, self.x, w.norm_next, self.next)
        return self.x


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=16)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=14336)
    ap.add_argument("--experts", type=int, default=0)
    ap.add_argument("--format", choices=("nvfp4", "mxfp4"), default="nvfp4")
    a = ap.parse_args()
    h = qg.gemm_create()
    w = Weights(h, a.hidden, a.inner, a.experts, qg.GEMM_NVFP4 if a.format == "nvfp4" else qg.GEMM_MXFP4)
    offsets = None
    if a.experts:
        # one expert a token, by random logits; the block's rows are the tokens in that order
        logits = torch.randn(a.tokens, a.experts, device="cuda")
        new = lambda *shape: torch.empty(*shape, dtype=torch.int32, device="cuda")  # noqa: E731
        ids, rows, offsets, weights = new(a.tokens, 1), new(a.tokens, 1), new(a.experts + 1), torch.empty(a.tokens, 1, device="cuda")
        workspace = qg.Workspace()
        check(qg.gemm_moe_route(h, qg.gemm_route_t(topk=1, scale=1.0), qg.ptr(logits), qg.row_major(logits), qg.ptr(ids), qg.ptr(weights),
                                qg.ptr(rows), qg.ptr(offsets), workspace.c, qg.current_stream()), "gemm_moe_route")
    b = Block(h, w, a.tokens, offsets)
    x = torch.randn(a.tokens, a.hidden, device="cuda").bfloat16()
    b.step(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step(x)
    for _ in range(3):
        graph.replay()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(50):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    check(qg.gemm_device_status(h, qg.current_stream()), "device status")
    print(f"{a.tokens} tokens, {a.hidden} -> {a.inner} -> {a.hidden}, {a.experts or 'no'} experts, {a.format}: "
          f"{start.elapsed_time(end) / 50 * 1e3:.1f} us a block")
    qg.gemm_destroy(h)


if __name__ == "__main__":
    main()
