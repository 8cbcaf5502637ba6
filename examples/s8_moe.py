"""A mixture-of-experts feed-forward layer in 8-bit integers, for a prompt or for
single tokens, out of the library's operators:

    choose every token's experts           gemm_moe_route
    place the tokens' rows by expert, int8 gemm_moe_dispatch
    up product + bias + GELU               gemm_run_s8_grouped
    quantise                               gemm_s8_quantize
    down product                           gemm_run_s8_grouped
    weighted sum, added to the residual    gemm_moe_combine

Weights are quantised once, one scale per output channel; activations have one
scale per row.  Run it for a time per step:

    python examples/s8_moe.py --tokens 16 --hidden 4096 --inner 14336 --experts 8 --topk 2
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
    """The layer's weights: int8 matrices [experts, out, in] with a scale per row, and
    the router's matrix."""

    def __init__(self, h, hidden, inner, experts, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
        self.hidden, self.inner, self.experts = hidden, inner, experts
        self.up, self.up_scale = self._quantize(h, new(experts, inner, hidden) * hidden ** -0.5)
        self.down, self.down_scale = self._quantize(h, new(experts, hidden, inner) * inner ** -0.5)
        self.up_bias = (0.1 * new(inner)).bfloat16()
        self.router = (new(experts, hidden) * hidden ** -0.5).bfloat16()
        self.router_bias = 0.01 * new(experts)  # for balance: it moves the choice, not the weights

    @staticmethod
    def _quantize(h, w):
        w = w.bfloat16()
        q = torch.empty(*w.shape[:2], -(-w.shape[2] // 16) * 16, dtype=torch.int8, device="cuda")[:, :, :w.shape[2]]
        s = torch.empty(w.shape[:2], device="cuda")
        check(qg.gemm_s8_quantize(h, qg.ptr(w), qg.row_major(w), qg.ptr(q), qg.row_major(q), qg.ptr(s), qg.current_stream()),
              "gemm_s8_quantize")
        return q, s


class Layer:
    """Buffers for `tokens` rows and the step itself."""

    def __init__(self, h, weights, tokens, topk):
        w = self.w = weights
        self.h, self.tokens, self.topk, rows = h, tokens, topk, tokens * topk
        new = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
        bf, i8, i32 = torch.bfloat16, torch.int8, torch.int32
        pad = lambda n: -(-n // 16) * 16  # noqa: E731  (rows of codes start every 16 bytes)
        self.workspace = qg.Workspace()
        self.logits = new(tokens, w.experts, dtype=bf)
        self.ids, self.weights, self.rows = new(tokens, topk, dtype=i32), new(tokens, topk), new(tokens, topk, dtype=i32)
        self.offsets = new(w.experts + 1, dtype=i32)
        self.x8, self.x_scale = new(rows, pad(w.hidden), dtype=i8)[:, :w.hidden], new(rows)
        self.mid = new(rows, w.inner, dtype=bf)
        self.mid8, self.mid_scale = new(rows, pad(w.inner), dtype=i8)[:, :w.inner], new(rows)
        self.out_rows, self.out = new(rows, w.hidden, dtype=bf), new(tokens, w.hidden, dtype=bf)
        self.route = qg.gemm_route_t(score=qg.GEMM_ROUTE_SIGMOID, topk=topk, renormalize=1, scale=1.0, bias=qg.ptr(w.router_bias))
        self.up_op = qg.gemm_op_t(epilogue=qg.GEMM_EPILOGUE_BIAS | qg.GEMM_EPILOGUE_GELU, bias=qg.ptr(w.up_bias), bias_type=qg.GEMM_BF16)

    def _product(self, op, a, a_scale, b, b_scale, d):
        check(qg.gemm_run_s8_grouped(self.h, op, 1.0, qg.ptr(a), qg.row_major(a), qg.ptr(a_scale), qg.ptr(b), qg.col_major_from_nk(b),
                                     qg.ptr(b_scale), 0.0, None, None, qg.ptr(d), qg.row_major(d), qg.ptr(self.offsets), self.w.experts,
                                     qg.current_stream()), "gemm_run_s8_grouped")

    def step(self, x):
        """x: [tokens, hidden] bf16 residual stream.  Returns the new one."""
        w, h, st = self.w, self.h, qg.current_stream()
        P, R = qg.ptr, qg.row_major
        # the router's logits: a plain product of the library
        check(qg.gemm_run(h, qg.gemm_op_t(), 1.0, P(x), R(x), None, None, P(w.router), qg.col_major_from_nk(w.router), None, None, 0.0, None,
                          None, P(self.logits), R(self.logits), self.workspace.c, st), "gemm_run")
        check(qg.gemm_moe_route(h, self.route, P(self.logits), R(self.logits), P(self.ids), P(self.weights), P(self.rows), P(self.offsets),
                                self.workspace.c, st), "gemm_moe_route")
        check(qg.gemm_moe_dispatch(h, P(x), R(x), P(self.rows), self.topk, P(self.x8), R(self.x8), P(self.x_scale), st), "gemm_moe_dispatch")
        self._product(self.up_op, self.x8, self.x_scale, w.up, w.up_scale, self.mid)
        check(qg.gemm_s8_quantize(h, P(self.mid), R(self.mid), P(self.mid8), R(self.mid8), P(self.mid_scale), st), "gemm_s8_quantize")
        self._product(qg.gemm_op_t(), self.mid8, self.mid_scale, w.down, w.down_scale, self.out_rows)
        check(qg.gemm_moe_combine(h, P(self.out_rows), R(self.out_rows), P(self.rows), P(self.weights), self.topk, 1.0, P(x), R(x), P(self.out),
                                  R(self.out), st), "gemm_moe_combine")
        return self.out


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=16)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=14336)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--topk", type=int, default=2)
    a = ap.parse_args()
    h = qg.gemm_create()
    layer = Layer(h, Weights(h, a.hidden, a.inner, a.experts), a.tokens, a.topk)
    x = torch.randn(a.tokens, a.hidden, device="cuda").bfloat16()
    layer.step(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(x)
    for _ in range(3):
        graph.replay()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(50):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    check(qg.gemm_device_status(h, qg.current_stream()), "device status")
    print(f"{a.tokens} tokens, {a.hidden} -> {a.inner} -> {a.hidden}, {a.topk} of {a.experts} experts, int8: "
          f"{start.elapsed_time(end) / 50 * 1e3:.1f} us a layer")
    qg.gemm_destroy(h)


if __name__ == "__main__":
    main()
