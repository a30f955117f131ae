"""The example's layer: prompts, then decode steps replayed from one graph.  Each
stage is checked against the oracle on the stage's own inputs, the cache byte for
byte after every step; eager steps give the same bits."""
import os
import sys

import numpy as np
import pytest
import torch

import oracle
import skinny_bit_gemm_amd as q
import workloads as wl
from oracle import attention as oa

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.lib()
    oracle.build()


def f32(t):
    return t.float().cpu().numpy()


class Checked:
    def __init__(self, ex, layer):
        self.ex, self.layer = ex, layer
        self.ref = oa.Cache(q.QLIN_FP8_DYNAMIC, ex.HK, ex.D, ex.PAGE, layer.cache.pages)
        for kv, (codes, scales) in enumerate(((layer.k, layer.ks), (layer.v, layer.vs))):      # whatever is there at first
            self.ref.codes[kv] = codes.cpu().numpy().reshape(self.ref.codes[kv].shape).copy()
            self.ref.scales[kv] = scales.cpu().numpy().reshape(self.ref.scales[kv].shape).copy()
        self.table = layer.table.cpu().numpy()

    def check(self, b, many):
        ex, layer = self.ex, self.layer
        HQ, HK, D = ex.HQ, ex.HK, ex.D
        qkv = f32(b.qkv).reshape(b.T, -1, D).astype(np.float64)
        at, table = b.position.cpu().numpy(), f32(layer.cos_sin)
        for out, heads, norm in ((b.q, qkv[:, :HQ], layer.q_norm), (b.k, qkv[:, HQ:HQ + HK], layer.k_norm)):
            y, size = oa.norm_rope(heads, f32(norm), 1e-6, table, at, D, 0)
            got = f32(out).reshape(y.shape)
            assert (np.abs(got - y) <= size * (D / 2 + 10) * U + np.abs(y) * 2.0 ** -8).all()
        offsets, lengths = b.offsets.cpu().numpy(), b.lengths.cpu().numpy()
        self.ref.append(offsets, lengths, self.table, f32(b.k).reshape(b.T, HK, D), f32(b.qkv).reshape(b.T, -1, D)[:, HQ + HK:])
        for kv, (codes, scales) in enumerate(((layer.k, layer.ks), (layer.v, layer.vs))):
            assert np.array_equal(codes.cpu().numpy().reshape(self.ref.codes[kv].shape), self.ref.codes[kv])
            got = scales.cpu().numpy().reshape(self.ref.scales[kv].shape)
            assert np.array_equal(got.view(np.uint32), self.ref.scales[kv].view(np.uint32))
        y, W, E, F = oa.attention(self.ref, offsets, lengths, self.table, f32(b.q).reshape(b.T, HQ, D), D ** -0.5)
        # the bound of one rounding to bf16, the probabilities' terms, and the sums of fewer than 512 tokens
        tol = E * U + W * ((2.0 ** -11 if many else 2.0 ** -16) + 700 * U) + F * 2.0 ** -21 + np.abs(y) * (2.0 ** -8 + 700 * U)
        assert (np.abs(f32(b.y).reshape(y.shape) - y) <= tol).all()
        # the o projection of what attention wrote
        qa, sa = oracle.quant_act(q.QLIN_FP8_DYNAMIC, b.y.view(torch.int16).cpu().numpy().view(np.uint16))
        assert np.array_equal(b.yq.cpu().numpy(), qa) and np.array_equal(b.ys.cpu().numpy(), sa)
        assert torch.isfinite(b.out.float()).all() and bool((b.out.float().abs().sum(1) > 0).all())


def test_prompts_then_replayed_steps():
    import attention_layer as ex
    lengths, context = [150, 3, 64, 300], 320
    layer = ex.Layer(len(lengths), context)
    checked = Checked(ex, layer)
    gen = torch.Generator(device="cuda").manual_seed(5)
    prompts = ex.Batch(layer, lengths, lengths)
    prompts.x.copy_(torch.randn(prompts.T, ex.HIDDEN, generator=gen, device="cuda"))
    layer.run(prompts)
    torch.cuda.synchronize()
    checked.check(prompts, True)
    decode = ex.Batch(layer, [1] * len(lengths), [n + 1 for n in lengths])
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = layer.capture(decode, stream)
    for step in range(4):
        decode.x.copy_(torch.randn(decode.T, ex.HIDDEN, generator=gen, device="cuda") * (1 + step))
        torch.cuda.synchronize()
        q.qlin_graph_launch(graph, stream)
        torch.cuda.synchronize()
        checked.check(decode, False)
        replayed = decode.out.clone()
        cache = [t.clone() for t in (layer.k, layer.v, layer.ks, layer.vs)]
        decode.out.zero_()
        layer.run(decode)                             # again and eagerly: the same tokens, the same bits
        torch.cuda.synchronize()
        assert torch.equal(decode.out.view(torch.int16), replayed.view(torch.int16))
        for t, was in zip((layer.k, layer.v, layer.ks, layer.vs), cache):
            assert torch.equal(t.view(torch.uint8), was.view(torch.uint8))
        decode.advance()
    q.qlin_graph_destroy(graph)


def test_the_example_runs():
    import attention_layer as ex
    argv, sys.argv = sys.argv, ["attention_layer.py", "3"]
    try:
        ex.main()
    finally:
        sys.argv = argv
    torch.cuda.synchronize()
    assert wl.SMALL_DENSE[0].N == (ex.HQ + 2 * ex.HK) * ex.D
