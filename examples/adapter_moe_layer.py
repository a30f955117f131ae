"""One decode step of a layer's second half, for requests with adapters of
their own: output projection and adapters, router, experts, residual.

    x  -> o projection (quantized)  + each request's low-rank adapter   = y
    y  -> router logits (quantized product, fp32 sums)
       -> top-8 of 128 experts, weights, rows grouped by expert
    y  -> quantized once, stored at its experts' rows
       -> gate and up of every expert in one grouped product
       -> silu(gate) x up, quantized
       -> down of every expert in one grouped product
       -> weighted sum of each token's rows, plus y

Every call takes its routing from device memory, so the step is captured into
one hipGraph and replayed with new activations, adapter ids and routing.  The
hidden size, the experts and the top-8 choice are the 128-expert workload's.

    python examples/adapter_moe_layer.py [tokens]
"""
from __future__ import annotations

import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import skinny_bit_gemm_amd as q  # noqa: E402
import workloads as wl  # noqa: E402

FMT = q.QLIN_FP8_DYNAMIC
PACKED = FMT | q.QLIN_PACKED_WEIGHTS
HIDDEN, INTER = wl.MOE_LAYERS[0].K, wl.MOE_LAYERS[1].K
EXPERTS, TOPK = wl.MOE_EXPERTS, wl.MOE_TOPK
ADAPTERS, RANK = 16, 16


def quantized(N, K, gen, batch=1):
    """Random weights [batch][N][K]: packed codes, scales."""
    dev = {"device": "cuda"}
    codes = torch.empty(batch, N, K, dtype=torch.uint8, **dev)
    scales = torch.empty(batch, N, **dev)
    for b in range(batch):
        w = torch.randn(N, K, generator=gen, **dev) * K ** -0.5
        q.qlin_quantize_weight(FMT, N, K, w, codes[b], scales[b])
    packed = torch.empty(batch * q.qlin_packed_weight_bytes(N, K), dtype=torch.uint8, **dev)
    q.qlin_pack_weight(batch, N, K, codes, packed)
    return {"N": N, "K": K, "codes": codes, "packed": packed, "scales": scales}


class Layer:
    """Weights, buffers and the step.  T is the batch's token count."""

    def __init__(self, T: int, seed: int = 0):
        dev, bf16, u8, i32 = {"device": "cuda"}, torch.bfloat16, torch.uint8, torch.int32
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.rows = T, T * TOPK
        self.o = quantized(HIDDEN, HIDDEN, gen)
        self.gate = quantized(EXPERTS, HIDDEN, gen)
        self.up = quantized(2 * INTER, HIDDEN, gen, EXPERTS)       # gate and up, one above the other
        self.down = quantized(HIDDEN, INTER, gen, EXPERTS)
        self.A = (torch.randn(ADAPTERS, RANK, HIDDEN, generator=gen, **dev) * HIDDEN ** -0.5).to(bf16)
        self.B = (torch.randn(ADAPTERS, HIDDEN, RANK, generator=gen, **dev) * RANK ** -0.5).to(bf16)
        self.ranks = torch.full((ADAPTERS,), RANK, dtype=i32, **dev)
        self.ranks[::3] = RANK // 2
        self.scales = torch.full((ADAPTERS,), 0.5, **dev)
        self.balance = torch.randn(EXPERTS, generator=gen, **dev) * 0.01
        self.router = q.make_router(EXPERTS, TOPK, q.QLIN_SCORE_SIGMOID, 8, 4, q.QLIN_GROUP_TOP2, 1, 2.5)
        # a step's inputs and buffers
        self.x = torch.zeros(T, HIDDEN, dtype=bf16, **dev)
        self.ids = torch.full((T,), -1, dtype=i32, **dev)
        self.xq, self.xs = torch.empty(T, HIDDEN, dtype=u8, **dev), torch.empty(T, **dev)
        self.shared = torch.empty(T, HIDDEN, dtype=bf16, **dev)
        self.y = torch.empty(T, HIDDEN, dtype=bf16, **dev)
        self.logits = torch.empty(T, EXPERTS, **dev)
        self.expert_ids, self.slots = (torch.empty(T, TOPK, dtype=i32, **dev) for _ in range(2))
        self.weights = torch.empty(T, TOPK, **dev)
        self.offsets = torch.empty(EXPERTS + 1, dtype=i32, **dev)
        self.row_token = torch.empty(self.rows, dtype=i32, **dev)
        self.eq, self.es = torch.zeros(self.rows, HIDDEN, dtype=u8, **dev), torch.zeros(self.rows, **dev)
        self.h, self.act32 = torch.zeros(self.rows, 2 * INTER, **dev), torch.empty(self.rows, INTER, **dev)
        self.act = torch.empty(self.rows, INTER, dtype=bf16, **dev)
        self.aq, self.as_ = torch.empty(self.rows, INTER, dtype=u8, **dev), torch.empty(self.rows, **dev)
        self.d = torch.zeros(self.rows, HIDDEN, dtype=bf16, **dev)
        self.out = torch.empty(T, HIDDEN, dtype=bf16, **dev)
        # split-K workspaces start as zeros and are left so; the others need no value
        zeroed = max(q.qlin_workspace_bytes(FMT, T, w["N"], w["K"]) for w in (self.o, self.gate))
        self.split_ws = torch.zeros(max(256, zeroed), dtype=u8, **dev)
        scratch = max(q.qlin_route_workspace_bytes(self.router, T),
                      q.qlin_lora_workspace_bytes(T, HIDDEN, HIDDEN, ADAPTERS, RANK))
        self.ws = torch.empty(max(256, scratch), dtype=u8, **dev)

    def step(self):
        """Enqueues the step on torch's current stream."""
        T, rows = self.T, self.rows
        q.qlin_linear(PACKED, T, HIDDEN, HIDDEN, self.x, HIDDEN, self.xq, self.xs, self.o["packed"], self.o["scales"],
                      self.shared, q.QLIN_OUT_BF16, None, self.split_ws)
        q.qlin_lora(T, HIDDEN, HIDDEN, ADAPTERS, RANK, self.x, HIDDEN, self.ids, self.A, self.B, self.ranks, self.scales,
                    self.shared, HIDDEN, self.y, HIDDEN, q.QLIN_OUT_BF16, self.ws)
        q.qlin_linear(PACKED, T, EXPERTS, HIDDEN, self.y, HIDDEN, self.xq, self.xs, self.gate["packed"],
                      self.gate["scales"], self.logits, q.QLIN_OUT_F32_ACC, None, self.split_ws)
        q.qlin_route(self.router, T, self.logits, EXPERTS, q.QLIN_OUT_F32_ACC, self.balance, self.expert_ids, self.weights,
                     self.offsets, self.row_token, self.slots, self.ws)
        q.qlin_dispatch_quantize(FMT, T, TOPK, HIDDEN, self.y, HIDDEN, self.slots, rows, self.eq, self.es)
        q.qlin_grouped_gemm(PACKED, EXPERTS, 2 * INTER, HIDDEN, self.offsets, rows, T, self.eq, self.es, self.up["packed"],
                            self.up["scales"], self.h, q.QLIN_OUT_F32_ACC)
        g, u = self.h[:, :INTER], self.h[:, INTER:]
        torch.sigmoid(g, out=self.act32)
        self.act.copy_(self.act32.mul_(g).mul_(u))
        q.qlin_quantize_act(FMT, rows, INTER, self.act, INTER, self.aq, self.as_)
        q.qlin_grouped_gemm(PACKED, EXPERTS, HIDDEN, INTER, self.offsets, rows, T, self.aq, self.as_, self.down["packed"],
                            self.down["scales"], self.d)
        q.qlin_combine(T, TOPK, HIDDEN, self.d, HIDDEN, q.QLIN_OUT_BF16, self.slots, self.weights, rows, self.y, HIDDEN,
                       self.out, HIDDEN)

    def capture(self, stream) -> int:
        with torch.cuda.stream(stream):
            self.step()              # once before: what is set up on first use is not part of a graph
            stream.synchronize()
            q.qlin_graph_begin(stream)
            self.step()
            return q.qlin_graph_end(stream)

    def set_inputs(self, seed: int):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.x.copy_(torch.randn(self.T, HIDDEN, generator=gen, device="cuda"))
        self.ids.copy_(torch.randint(-1, ADAPTERS, (self.T,), generator=gen, device="cuda"))


def main():
    T = int(sys.argv[1]) if len(sys.argv) > 1 else 16
    layer = Layer(T)
    layer.set_inputs(1)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    graph = layer.capture(stream)
    for seed in (2, 3):
        layer.set_inputs(seed)
        torch.cuda.synchronize()
        q.qlin_graph_launch(graph, stream)
        torch.cuda.synchronize()
        used = int((layer.offsets[1:] > layer.offsets[:-1]).sum())
        print(f"{T} tokens: {used} of {EXPERTS} experts in use, |out| {layer.out.float().abs().mean():.4f}, "
              f"first token's experts {layer.expert_ids[0].tolist()}")
    n = 200
    t = time.perf_counter()
    for _ in range(n):
        q.qlin_graph_launch(graph, stream)
    torch.cuda.synchronize()
    print(f"{(time.perf_counter() - t) / n * 1e6:.1f} us a step (graph replay)")
    q.qlin_graph_destroy(graph)


if __name__ == "__main__":
    main()
