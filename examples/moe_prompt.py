"""A routed-expert layer on a prompt with 4-bit weights and 4-bit activations.

Experts with MXFP4 weights [inter, hidden] (gate, up) and [hidden, inter] (down); every
token's hidden vector goes to its top-k experts:

    sort      the (token, expert) pairs into expert order
    quantise  x, gathered into that order on the way, to MXFP4
    gate, up  each expert's rows with its matrices
    act       silu(gate) * up, quantised again
    down      each expert's rows with its matrix
    combine   back to token order with the route weights

Seven launches, nothing allocated between them, so the layer can be captured in a graph.
`python examples/moe_prompt.py` makes a layer with random weights, runs it, and prints its
time and how far it is from the same layer with FP32 activations (mxfp4_moe_gate_up /
mxfp4_moe_down, built for few tokens per expert): the difference is the 4-bit rounding of the
activations.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_dequant_matmul_gb300 as mx  # noqa: E402


def quantise(x, row_of=None, rows=None):
    """Rows of a 2-D tensor (or its rows row_of) as an MXFP4 matrix."""
    x_rows, cols = x.shape
    rows = x_rows if rows is None else rows
    out = torch.empty(mx.mxfp4_nbytes(rows, cols), dtype=torch.uint8, device=x.device)
    mx.mxfp4_quant(x, x_rows, cols, x.stride(0), row_of, rows, out)
    return out


def make_bank(n_experts, rows, cols, scale):
    """n_experts random matrices, quantised one after the other into one bank."""
    size = mx.mxfp4_nbytes(rows, cols)
    bank = torch.empty(n_experts * size, dtype=torch.uint8, device="cuda")
    for e in range(n_experts):
        w = scale * torch.randn(rows, cols, device="cuda")
        mx.mxfp4_quant(w, rows, cols, cols, None, rows, bank[e * size:(e + 1) * size])
    return bank


class MoePrompt:
    """The layer's weights and the buffers of up to max_tokens tokens."""

    def __init__(self, gate, up, down, n_experts, hidden, inter, top_k, max_tokens,
                 dtype=torch.bfloat16):
        if dtype not in (torch.float32, torch.bfloat16):   # what the products write
            raise ValueError(f"buffers of {dtype}: float32 or bfloat16")
        self.gate, self.up, self.down = gate, up, down
        self.n_experts, self.hidden, self.inter, self.top_k = n_experts, hidden, inter, top_k
        self.max_tokens, pairs = max_tokens, max_tokens * top_k
        i32 = dict(dtype=torch.int32, device="cuda")
        self.token_at, self.pos_of = torch.empty(pairs, **i32), torch.empty(pairs, **i32)
        self.offsets = torch.empty(n_experts + 1, **i32)
        u8 = dict(dtype=torch.uint8, device="cuda")
        self.xq = torch.empty(mx.mxfp4_nbytes(pairs, hidden), **u8)
        self.aq = torch.empty(mx.mxfp4_nbytes(pairs, inter), **u8)
        self.g, self.u = (torch.empty(pairs, inter, dtype=dtype, device="cuda") for _ in range(2))
        self.o = torch.empty(pairs, hidden, dtype=dtype, device="cuda")

    def __call__(self, x, expert_ids, route_w, y):
        """x [tokens, hidden] -> y [tokens, hidden] of the buffers' type; expert_ids [tokens, top_k]
        int32 (a pair with an id outside the experts adds nothing), route_w [tokens, top_k] float."""
        tokens, pairs = x.shape[0], x.shape[0] * self.top_k
        if tokens > self.max_tokens:
            raise ValueError(f"{tokens} tokens, room for {self.max_tokens}")
        if x.shape[1] != self.hidden or x.stride(1) != 1:
            raise ValueError(f"x {tuple(x.shape)}, strides {x.stride()}: rows of {self.hidden}")
        for t, shape in ((expert_ids, (tokens, self.top_k)), (route_w, (tokens, self.top_k)),
                         (y, (tokens, self.hidden))):
            if tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"a contiguous {shape} instead of {tuple(t.shape)}, strides "
                                 f"{t.stride()}")
        mx.mxfp4_moe_sort(expert_ids, tokens, self.top_k, self.n_experts, self.token_at,
                          self.pos_of, self.offsets)
        mx.mxfp4_quant(x, tokens, self.hidden, x.stride(0), self.token_at, pairs, self.xq)
        for bank, out in ((self.gate, self.g), (self.up, self.u)):
            mx.mxfp4_moe_mm_mx(bank, self.n_experts, self.inter, self.hidden, self.xq, pairs,
                               self.offsets, out)
        mx.mxfp4_swiglu_quant(self.g, self.u, pairs, self.inter, self.inter, self.aq)
        mx.mxfp4_moe_mm_mx(self.down, self.n_experts, self.hidden, self.inter, self.aq, pairs,
                           self.offsets, self.o)
        mx.mxfp4_moe_combine(self.o, tokens, self.top_k, self.hidden, self.pos_of, route_w, y)
        return y


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--tokens", type=int, default=2048)
    p.add_argument("--experts", type=int, default=64)
    p.add_argument("--hidden", type=int, default=2880)
    p.add_argument("--inter", type=int, default=2880)
    p.add_argument("--top-k", type=int, default=4)
    a = p.parse_args()
    torch.manual_seed(0)
    gate, up = (make_bank(a.experts, a.inter, a.hidden, a.hidden ** -0.5) for _ in range(2))
    down = make_bank(a.experts, a.hidden, a.inter, a.inter ** -0.5)
    layer = MoePrompt(gate, up, down, a.experts, a.hidden, a.inter, a.top_k, a.tokens)
    x = torch.randn(a.tokens, a.hidden, device="cuda").bfloat16()
    logits = torch.randn(a.tokens, a.experts, device="cuda")
    route_w, ids = torch.softmax(logits, -1).topk(a.top_k)
    route_w, ids = (route_w / route_w.sum(-1, keepdim=True)).contiguous(), ids.int().contiguous()
    y = torch.empty_like(x)
    layer(x, ids, route_w, y)
    torch.cuda.synchronize()

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(x, ids, route_w, y)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for _ in range(3):
        graph.replay()
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    us = start.elapsed_time(end) / 20 * 1e3
    flops = 6 * a.tokens * a.top_k * a.hidden * a.inter
    print(f"{a.tokens} tokens: {us:.1f} us a layer, {flops / us / 1e6:.0f} TFLOP/s")

    n = min(a.tokens, 64)                     # the FP32-activation layer, on the first tokens
    act = torch.empty(n * a.top_k * a.inter, device="cuda")
    ref = torch.empty(n, a.hidden, device="cuda")
    ws = torch.empty(mx.mxfp4_moe_workspace_bytes(a.experts, n, a.top_k, a.hidden, a.inter),
                     dtype=torch.uint8, device="cuda")
    xf = x[:n].float().contiguous()
    mx.mxfp4_moe_gate_up(gate, up, a.experts, a.hidden, a.inter, xf, n, a.top_k, ids, act, ws)
    mx.mxfp4_moe_down(down, a.experts, a.hidden, a.inter, act, n, a.top_k, ids, route_w, ref, ws)
    d = (y[:n].float() - ref).norm() / ref.norm()
    print(f"against FP32 activations: {d.item():.3f} of the result's norm")


if __name__ == "__main__":
    main()
