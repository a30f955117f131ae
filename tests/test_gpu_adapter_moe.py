"""The calls together, as examples/adapter_moe_layer.py runs them: each stage
of a step against the oracle on that stage's own inputs, eagerly and in
replays of one graph after the routing has changed."""
import os
import sys

import numpy as np
import pytest
import torch

import oracle
import skinny_bit_gemm_amd as q
from oracle import rows as orows

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.lib()
    oracle.build()


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def f64(t):
    return t.double().cpu().numpy()


def check_stages(L, ex):
    """Every stage from the device's own inputs of it."""
    T, FMT = L.T, ex.FMT
    _, _, ref = oracle.linear(FMT, bits(L.x), L.o["codes"][0].cpu().numpy(), L.o["scales"][0].cpu().numpy())
    ok, worst = oracle.tolerance_ok(f64(L.shared), ref)
    assert ok, f"o projection ({worst:.3g})"

    y, of_v, of_terms = orows.lora(f64(L.x), L.ids.cpu().numpy(), f64(L.A), f64(L.B), L.ranks.cpu().numpy(),
                                   L.scales.cpu().numpy(), f64(L.shared))
    tol = 4 * (np.sqrt(ex.HIDDEN) + 8) * 2.0 ** -24 * of_terms + 2.0 ** -16 * of_v
    assert (np.abs(f64(L.y) - y) <= tol + 2.0 ** -8 * (np.abs(y) + tol) + 1e-37).all(), "adapters"

    ids, w, off, rows, slots = orows.route(f64(L.logits), ex.TOPK, orows.SIGMOID, f64(L.balance), 8, 4, orows.TOP2, 1, 2.5)
    assert np.array_equal(L.expert_ids.cpu().numpy(), ids) and np.array_equal(L.offsets.cpu().numpy(), off)
    assert np.array_equal(L.row_token.cpu().numpy(), rows) and np.array_equal(L.slots.cpu().numpy(), slots)
    assert np.allclose(L.weights.cpu().numpy(), w, rtol=1e-5, atol=0)

    qa, sa = oracle.quant_act(FMT, bits(L.y))
    assert np.array_equal(L.eq.cpu().numpy(), qa.view(np.uint8)[rows]), "dispatched codes"
    assert np.array_equal(L.es.cpu().numpy(), sa[rows]), "dispatched scales"

    for name, w_, codes, scales, out in (("gate and up", L.up, L.eq, L.es, L.h), ("down", L.down, L.aq, L.as_, L.d)):
        used = np.unique(ids)
        ref = np.zeros(tuple(out.shape))
        for e in used:
            r = slice(off[e], off[e + 1])
            ref[r] = oracle.gemm(FMT, codes.cpu().numpy()[r], scales.cpu().numpy()[r], w_["codes"][e].cpu().numpy(),
                                 w_["scales"][e].cpu().numpy())
        ok, worst = oracle.tolerance_ok(f64(out), ref)
        assert ok, f"{name} ({worst:.3g})"

    ref, size = orows.combine(f64(L.d), slots, f64(L.weights), f64(L.y))
    tol = (ex.TOPK + 2) * 2.0 ** -24 * size
    assert (np.abs(f64(L.out) - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol) + 1e-37).all(), "combine"


@pytest.mark.parametrize("T", [1, 13])
def test_step_and_graph_replays(T):
    import adapter_moe_layer as ex
    L = ex.Layer(T, seed=5)
    L.set_inputs(1)
    L.step()
    torch.cuda.synchronize()
    check_stages(L, ex)
    stream = torch.cuda.Stream()
    graph = L.capture(stream)
    torch.cuda.synchronize()
    for seed in (2, 3, 2):
        L.set_inputs(seed)
        L.out.zero_()
        torch.cuda.synchronize()
        q.qlin_graph_launch(graph, stream)
        torch.cuda.synchronize()
        check_stages(L, ex)
    q.qlin_graph_destroy(graph)
