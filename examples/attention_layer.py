"""A layer's first half over an 8-bit cache: prompts, then decode steps.

    x -> qkv projection (quantized)
      -> norm of each query and key head, rotation by position
      -> keys and values quantized into the pages of their sequences
      -> attention of the new tokens over all cached ones
      -> o projection (quantized)

A prompt of every sequence goes through it eagerly; a decode step (one token
for each sequence) is captured into one hipGraph, which is replayed while lengths,
positions and page tables move on in device memory.  Sizes are those of the
hidden-2048 workload: 16 query and 8 key heads, 128 wide.

    python examples/attention_layer.py [sequences]
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
QKV, O = wl.SMALL_DENSE[0], wl.SMALL_DENSE[1]
HIDDEN, D = QKV.K, 128
HQ = O.K // D
HK = (QKV.N // D - HQ) // 2
PAGE = 64


def quantized(layer, gen):
    """Random weights of a linear layer: packed codes, scales."""
    dev = {"device": "cuda"}
    w = torch.randn(layer.N, layer.K, generator=gen, **dev) * layer.K ** -0.5
    codes, scales = torch.empty(layer.N, layer.K, dtype=torch.uint8, **dev), torch.empty(layer.N, **dev)
    q.qlin_quantize_weight(FMT, layer.N, layer.K, w, codes, scales)
    packed = torch.empty(q.qlin_packed_weight_bytes(layer.N, layer.K), dtype=torch.uint8, **dev)
    q.qlin_pack_weight(1, layer.N, layer.K, codes, packed)
    return {"N": layer.N, "K": layer.K, "packed": packed, "scales": scales}


def rope_table(positions, base=1e6):
    """[positions][D] fp32: cosines, then sines, of angles taken in 64 bits."""
    turn = base ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * turn
    return torch.cat([angle.cos(), angle.sin()], 1).float().cuda()


class Batch:
    """A call's tokens: buffers of T rows, and where they belong."""

    def __init__(self, layer, new, lengths):
        """new: tokens of each sequence; lengths: of the sequences, with them."""
        dev, bf16, i32 = {"device": "cuda"}, torch.bfloat16, torch.int32
        T, B = int(sum(new)), len(new)
        self.T = T
        self.x = torch.zeros(T, HIDDEN, dtype=bf16, **dev)
        self.xq, self.xs = torch.empty(T, HIDDEN, dtype=torch.uint8, **dev), torch.empty(T, **dev)
        self.qkv = torch.empty(T, QKV.N, dtype=bf16, **dev)
        self.q, self.k = torch.empty(T, HQ * D, dtype=bf16, **dev), torch.empty(T, HK * D, dtype=bf16, **dev)
        self.y = torch.empty(T, HQ * D, dtype=bf16, **dev)
        self.yq, self.ys = torch.empty(T, HQ * D, dtype=torch.uint8, **dev), torch.empty(T, **dev)
        self.out = torch.empty(T, HIDDEN, dtype=bf16, **dev)
        self.offsets = torch.tensor([sum(new[:i]) for i in range(B + 1)], dtype=i32, **dev)
        self.lengths = torch.tensor(list(lengths), dtype=i32, **dev)
        self.position = torch.tensor([l - n + i for n, l in zip(new, lengths) for i in range(n)], dtype=i32, **dev)
        self.sequences = q.make_sequences(B, T, self.offsets, self.lengths, layer.table, layer.table.shape[1],
                                          layer.context)
        need = q.qlin_cache_attention_workspace_bytes(layer.attention, layer.cache, self.sequences)
        self.work = torch.empty(max(256, need), dtype=torch.uint8, **dev)
        split = max(q.qlin_workspace_bytes(FMT, T, w["N"], w["K"]) for w in (layer.qkv, layer.o))
        self.split_work = torch.zeros(max(256, split), dtype=torch.uint8, **dev)   # zeros, and left so

    def advance(self):
        """The next decode step: a token more in every sequence."""
        self.lengths += 1
        self.position += 1


class Layer:
    def __init__(self, sequences, context, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        dev = {"device": "cuda"}
        self.context = context
        self.qkv, self.o = quantized(QKV, gen), quantized(O, gen)
        self.q_norm, self.k_norm = (1 + 0.2 * torch.randn(D, generator=gen, **dev) for _ in range(2))
        self.cos_sin = rope_table(context)
        self.rope = q.make_rope(HQ, HK, D, D, context)
        self.attention = q.make_attention(HQ, D ** -0.5)
        width = -(-context // PAGE)
        pages = sequences * width
        sizes = q.qlin_cache_bytes(q.make_cache(FMT, HK, D, PAGE, pages))
        self.k, self.v = (torch.empty(sizes[0], dtype=torch.uint8, **dev) for _ in range(2))
        self.ks, self.vs = (torch.empty(sizes[1] // 4, **dev) for _ in range(2))
        self.cache = q.make_cache(FMT, HK, D, PAGE, pages, self.k, self.v, self.ks, self.vs)
        self.table = torch.randperm(pages, generator=gen, **dev).to(torch.int32).view(sequences, width)

    def run(self, b: Batch, stream=None):
        """Enqueues the layer on `stream` (torch's current one)."""
        T, ld = b.T, QKV.N
        q.qlin_linear(PACKED, T, QKV.N, HIDDEN, b.x, HIDDEN, b.xq, b.xs, self.qkv["packed"], self.qkv["scales"], b.qkv,
                      q.QLIN_OUT_BF16, None, b.split_work, stream=stream)
        keys, values = b.qkv[:, HQ * D:], b.qkv[:, (HQ + HK) * D:]
        q.qlin_norm_rope(self.rope, T, b.qkv, ld, keys, ld, q.QLIN_OUT_BF16, self.q_norm, self.k_norm, self.cos_sin,
                         b.position, b.q, HQ * D, b.k, HK * D, stream=stream)
        q.qlin_cache_append(self.cache, b.sequences, b.k, HK * D, values, ld, stream=stream)
        q.qlin_cache_attention(self.attention, self.cache, b.sequences, b.q, HQ * D, b.y, HQ * D, q.QLIN_OUT_BF16, b.work,
                               stream=stream)
        q.qlin_linear(PACKED, T, HIDDEN, HQ * D, b.y, HQ * D, b.yq, b.ys, self.o["packed"], self.o["scales"], b.out,
                      q.QLIN_OUT_BF16, None, b.split_work, stream=stream)

    def capture(self, b: Batch, stream) -> int:
        q.qlin_graph_begin(stream)
        self.run(b, stream)
        return q.qlin_graph_end(stream)


def main():
    B = int(sys.argv[1]) if len(sys.argv) > 1 else 16
    context, steps = 4096, 64
    layer = Layer(B, context)
    gen = torch.Generator(device="cuda").manual_seed(1)
    lengths = [context - steps - 1 - 37 * i for i in range(B)]
    prompts = Batch(layer, lengths, lengths)
    prompts.x.copy_(torch.randn(prompts.T, HIDDEN, generator=gen, device="cuda"))
    torch.cuda.synchronize()
    t = time.perf_counter()
    layer.run(prompts)
    torch.cuda.synchronize()
    print(f"{B} prompts, {prompts.T} tokens: {(time.perf_counter() - t) * 1e3:.2f} ms, |out| {prompts.out.float().abs().mean():.4f}")
    decode = Batch(layer, [1] * B, [n + 1 for n in lengths])
    decode.x.copy_(torch.randn(B, HIDDEN, generator=gen, device="cuda"))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = layer.capture(decode, stream)
    with torch.cuda.stream(stream):
        for i in range(steps):
            q.qlin_graph_launch(graph, stream)
            if i + 1 < steps:
                decode.advance()
    torch.cuda.synchronize()
    print(f"after {steps} steps the longest sequence has {int(decode.lengths.max())} tokens, "
          f"|out| {decode.out.float().abs().mean():.4f}")
    n = 200
    t = time.perf_counter()
    for _ in range(n):
        q.qlin_graph_launch(graph, stream)         # the last step again: it stores the same tokens
    torch.cuda.synchronize()
    print(f"{(time.perf_counter() - t) / n * 1e6:.1f} us a step (graph replay)")
    q.qlin_graph_destroy(graph)


if __name__ == "__main__":
    main()
