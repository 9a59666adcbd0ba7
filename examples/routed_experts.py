"""One routed-expert layer of a multi-adapter serving step, every operator on
the GPU and nothing read back to the host:

    router logits (+ router LoRA) -> experts and weights -> expert-sorted rows
    -> rows in MXFP4 -> gate/up product (+ experts' LoRA) -> silu(gate) * up in
    MXFP4 -> down product (+ experts' LoRA) -> weighted sum onto the residual

    python examples/routed_experts.py [--tokens 256] [--experts 8] [--top-k 2]
        [--hidden 4096] [--inter 14336] [--slots 32]

prints the step's time, eager and replayed as a HIP graph. Random weights and
adapters.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import adapter_lora_serving_amd as L  # noqa: E402


class RoutedExperts:
    """The weights and adapters of one layer: a bf16 router, MXFP4 experts
    (gate and up stacked), a LoRA per slot on the router and per (expert,
    slot) on both expert projections."""

    def __init__(self, hidden, inter, experts, slots, top_k, rank=16, seed=0, device="cuda:0"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def draw(*shape, std):
            return (torch.randn(*shape, device=device, generator=g) * std).bfloat16()

        self.hidden, self.inter, self.experts = hidden, inter, experts
        self.slots, self.top_k = slots, top_k
        self.router = draw(experts, hidden, std=2 / math.sqrt(hidden))
        self.gate_up = self._held(draw, 2 * inter, hidden)
        self.down = self._held(draw, hidden, inter)
        pool = experts * slots
        self.ranks = torch.randint(0, rank + 1, (slots,), device=device, generator=g,
                                   dtype=torch.int32)
        self.scalings = torch.full((slots,), 0.5, device=device)
        self.pool_ranks = self.ranks.repeat(experts)
        self.pool_scalings = self.scalings.repeat(experts)

        def lora(entries, out, in_features):
            return (draw(entries, rank, in_features, std=1 / math.sqrt(in_features)),
                    draw(entries, out, rank, std=1 / math.sqrt(rank)))

        self.router_lora = lora(slots, experts, hidden)
        a, b = lora(pool, 2 * inter, hidden)
        self.gate_up_lora = (torch.cat([a, a.flip(0)], 1).contiguous(), b)   # a slice each
        self.down_lora = lora(pool, hidden, inter)

    def _held(self, draw, out, in_features):
        parts = [L.quantize_mxfp4(draw(out, in_features, std=1 / math.sqrt(in_features)))
                 for _ in range(self.experts)]
        return L.MXFP4(*(torch.stack(p) for p in zip(*parts)))

    def step(self, x, residual, token_slot):
        """The layer's output for tokens x [T, hidden], each with its adapter
        slot (-1: none), and every tensor on the way."""
        t = {}
        # the router's product by torch (its width is a few dozen columns)
        t["base_logits"] = x @ self.router.t()
        t["logits"] = t["base_logits"].clone()
        L.apply_linear_from_slots_(x, t["logits"], *self.router_lora, token_slot, self.ranks,
                                   self.scalings, (self.experts,))
        t["routing"] = L.route_experts(t["logits"], self.top_k)
        t["sorted"] = L.expert_rows(t["routing"].ids, self.experts, token_slot)
        offsets, row_slot = t["sorted"].offsets, t["sorted"].row_slot
        t["rows"], t["x"] = L.gather_quantize_mxfp4(x, t["sorted"].row_token)
        t["base_gate_up"] = L.mxfp4_expert_linear(t["x"], self.gate_up, offsets)
        t["gate_up"] = t["base_gate_up"].clone()
        addr = L.apply_linear_from_experts_(t["rows"], t["gate_up"], *self.gate_up_lora, row_slot,
                                            offsets, self.experts, self.slots, self.pool_ranks,
                                            self.pool_scalings, (self.inter, self.inter))
        t["act"], t["h"] = L.silu_mul_quantize_mxfp4(t["gate_up"])
        t["base_down"] = L.mxfp4_expert_linear(t["h"], self.down, offsets)
        t["down"] = t["base_down"].clone()
        L.apply_linear_(t["act"], t["down"], *self.down_lora, addr, self.pool_ranks,
                        self.pool_scalings, (self.hidden,))
        t["y"] = L.combine_experts(t["down"], t["sorted"].positions, t["routing"].weights,
                                   residual=residual)
        return t


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, v in (("tokens", 256), ("experts", 8), ("top-k", 2), ("hidden", 4096),
                    ("inter", 14336), ("slots", 32), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=v)
    a = ap.parse_args()
    layer = RoutedExperts(a.hidden, a.inter, a.experts, a.slots, a.top_k)
    g = torch.Generator(device="cuda:0")
    g.manual_seed(1)
    x = torch.randn(a.tokens, a.hidden, device="cuda:0", generator=g).bfloat16()
    residual = torch.randn(a.tokens, a.hidden, device="cuda:0", generator=g).bfloat16()
    slot = torch.randint(-1, a.slots, (a.tokens,), device="cuda:0", generator=g,
                         dtype=torch.int32)

    def timed(f):
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        for _ in range(a.steps):
            f()
        end.record()
        torch.cuda.synchronize()
        return begin.elapsed_time(end) / a.steps * 1e3

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        for _ in range(3):
            eager = layer.step(x, residual, slot)["y"]
        torch.cuda.synchronize()
        t_eager = timed(lambda: layer.step(x, residual, slot))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            y = layer.step(x, residual, slot)["y"]
        graph.replay()
        torch.cuda.synchronize()
        same = torch.equal(y, eager)
        t_graph = timed(graph.replay)
    print(f"{a.tokens} tokens, top-{a.top_k} of {a.experts} experts, {a.hidden} x {a.inter}, "
          f"{a.slots} adapter slots: {t_eager:.1f} us a step, {t_graph:.1f} us as a graph "
          f"(same output: {same})")


if __name__ == "__main__":
    main()
