"""A feed-forward block with its weights in MXFP4: a projection, a router and a mixture-of-experts layer.

    h  = x + W x                       Mxfp4Weight.gemm (decode) or gemm_mx on quantized x (prefill)
    l  = R h                           router logits, Int8Weight.gemm
    y  = h + sum of top-k experts(h)   moe_layer, the residual in the same call

The prompt goes through once; then tokens follow one at a time from a graph that was captured once and is
replayed.  Weights and inputs are random; the printed error is against the same block in float32 on the
dequantized weights.

    python examples/mxfp4_moe_block.py [--hidden 4096 --inner 14336 --experts 8 --topk 2 --prompt 48 --tokens 32]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from weight_only_quantized_int8_amd import Int8Weight, Mxfp4Weight, moe_layer  # noqa: E402


class Block:
    def __init__(self, hidden: int, inner: int, experts: int, topk: int, seed: int = 0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def dense(n, k, gain=1.0):
            w = torch.randn((n, k), generator=g, device="cuda", dtype=torch.float32)
            return (w * (gain / k ** 0.5)).bfloat16()

        self.experts, self.topk = experts, topk
        self.proj = Mxfp4Weight.quantize(dense(hidden, hidden))
        self.router = Int8Weight.quantize(dense(experts, hidden, 2.0), 64)
        self.gate, self.up = (Mxfp4Weight.quantize(dense(experts * inner, hidden)) for _ in range(2))
        self.down = Mxfp4Weight.quantize(dense(experts * hidden, inner))

    def _experts(self, h: torch.Tensor) -> torch.Tensor:
        logits = self.router.gemm(h)
        return moe_layer(self.gate, self.up, self.down, self.experts, h, logits, self.topk, x_resid=h)

    def prefill(self, x: torch.Tensor) -> torch.Tensor:
        return self._experts(x + self.proj.gemm_mx(Mxfp4Weight.quantize(x)))

    def decode(self, x: torch.Tensor) -> torch.Tensor:
        return self._experts(x + self.proj.gemm(x))

    def plain(self, x: torch.Tensor, prefill: bool) -> torch.Tensor:
        """The same in float32, expert by expert."""
        W = self.proj.dequantize_to().float()
        xq = Mxfp4Weight.quantize(x).dequantize_to() if prefill else x
        h = (x + (xq.float() @ W.t()).bfloat16()).float()
        logits = (h @ self.router.dequantize_to().float().t()).bfloat16().float()
        top, ids = logits.topk(self.topk, dim=1)
        p = torch.softmax(top, dim=1)
        gate, up, down = (w.dequantize_to().view(self.experts, -1, w.k) for w in (self.gate, self.up, self.down))
        y = h.clone()
        for t in range(h.shape[0]):
            for j in range(self.topk):
                e = int(ids[t, j])
                a = torch.nn.functional.silu(gate[e].float() @ h[t]) * (up[e].float() @ h[t])
                y[t] += p[t, j] * (down[e].float() @ a)
        return y


def run(hidden=4096, inner=14336, experts=8, topk=2, prompt=48, tokens=32):
    """Relative errors of the prefill and of a decoded token, and microseconds a replayed token."""
    block = Block(hidden, inner, experts, topk)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn((prompt, hidden), generator=g, device="cuda").bfloat16()

    def error(y, ref):
        return float((y.float() - ref).norm() / ref.norm())

    y = block.prefill(x)
    pre = error(y, block.plain(x, True))

    token = x[:1].clone()
    block.decode(token)  # everything is loaded before the capture
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        out = block.decode(token)
    torch.cuda.synchronize()
    dec = 0.0
    for t in range(3):  # replays with other tokens
        token.copy_(x[t:t + 1])
        graph.replay()
        dec = max(dec, error(out, block.plain(token, False)))
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(tokens):
        graph.replay()
    torch.cuda.synchronize()
    return pre, dec, (time.perf_counter() - start) / tokens * 1e6


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("hidden", 4096), ("inner", 14336), ("experts", 8), ("topk", 2), ("prompt", 48), ("tokens", 32)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    pre, dec, us = run(a.hidden, a.inner, a.experts, a.topk, a.prompt, a.tokens)
    print(f"prefill of {a.prompt} tokens: relative error {pre:.4f}")
    print(f"decode: relative error {dec:.4f}, {us:.1f} us a token")


if __name__ == "__main__":
    main()
