"""Routing, dispatch and combine on the GPU against the 64-bit oracle: ids,
offsets, rows and slots equal, codes and scales equal, weights and sums
within the rounding errors that their fp32 arithmetic can make."""
import numpy as np
import pytest
import torch

import oracle
import skinny_bit_gemm_amd as q
import workloads as wl
from oracle import rows as orows

pytestmark = pytest.mark.gpu

from _gpu import DEV, as_u8, check_guards, guarded, to_dev, to_dev_bf16  # noqa: E402

INF, NAN = np.inf, np.nan
SOFT, SIG = q.QLIN_SCORE_SOFTMAX, q.QLIN_SCORE_SIGMOID
BF16, F32 = q.QLIN_OUT_BF16, q.QLIN_OUT_F32_ACC
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.lib()
    oracle.build()


def logits_for(T, E, seed, bf16, masked=0.0, std=1.5):
    """fp32 logits (values of bf16 where they will be stored so)."""
    rng = np.random.default_rng([11, T, E, seed])
    l = rng.normal(0.0, std, size=(T, E)).astype(np.float32)
    l[rng.random((T, E)) < masked] = -INF
    return l if not bf16 else wl.bf16_bits_to_f32(to_bits(l))


def to_bits(l):
    """bf16 bit patterns, infinities and NaN kept."""
    l = np.asarray(l, dtype=np.float32)
    bits = wl._to_bf16_bits(np.where(np.isfinite(l), l, 0.0))
    bits[np.isposinf(l)], bits[np.isneginf(l)], bits[np.isnan(l)] = 0x7F80, 0xFF80, 0x7FC0
    return bits


def device_logits(l, bf16, ld):
    T, E = l.shape
    if bf16:
        wide = np.full((T, ld), 0x7F00, dtype=np.uint16)      # large values past the experts
        wide[:, :E] = to_bits(l)
        return to_dev_bf16(wide)
    wide = np.full((T, ld), 1e30, dtype=np.float32)
    wide[:, :E] = l
    return to_dev(wide)


def run_route(router, logits, T, ld, lt, bias):
    E, k = router.experts, router.topk
    ids, slots = guarded((T, k), torch.int32, -7), guarded((T, k), torch.int32, -7)
    w = guarded((T, k), torch.float32, -7.0)
    off, rows = guarded((E + 1,), torch.int32, -7), guarded((T * k,), torch.int32, -7)
    work = guarded((max(16, q.qlin_route_workspace_bytes(router, T)),), torch.uint8, 0xEE)
    bd = None if bias is None else to_dev(np.asarray(bias, dtype=np.float32))
    q.qlin_route(router, T, logits, ld, lt, bd, ids, w, off, rows, slots, work)
    torch.cuda.synchronize()
    check_guards(ids, slots, w, off, rows, work, what=f"qlin_route T={T} E={E} k={k}")
    return [v.cpu().numpy() for v in (ids, w, off, rows, slots)]


def check_route(l, bf16=False, bias=None, ld=None, **r):
    T, E = l.shape
    r = {"topk": min(8, E), **r}
    router = q.make_router(E, **r)
    ld = E if ld is None else ld
    print(f"[route] T={T} E={E} bf16={bf16} bias={bias is not None} ld={ld} {r}", flush=True)
    got = run_route(router, device_logits(l, bf16, ld), T, ld, BF16 if bf16 else F32, bias)
    scale = np.float32(r.get("scale", 1.0))
    want = orows.route(l, r["topk"], r.get("score", SOFT), bias, r.get("groups", 1), r.get("topk_groups", 1),
                       r.get("group_score", 0), r.get("renormalize", 1), scale)
    for name, g, x in zip(("ids", "offsets", "rows", "slots"), [got[0]] + got[2:], [want[0]] + list(want[2:])):
        assert np.array_equal(g, x), f"{name} differ"
    # a weight: the difference l - top (rounded: |l - top| U, an exponent's absolute error is the result's
    # relative one), an exponential (1 ulp is 2 U), a sum of at most 1024 positive terms through 16 + 6 levels,
    # a division and a product
    finite = np.where(np.isfinite(l), np.clip(l, -100.0, 100.0), 0.0)
    spread = 2.0 * np.abs(finite).max(initial=0.0)
    err = np.abs(got[1].astype(np.float64) - want[1])
    assert (err <= (2 * spread + 32) * U * np.abs(want[1]) + 1e-37).all(), f"weights off by {err.max()}"
    return got


@pytest.mark.parametrize("T", [1, 15, 16, 17, 64, 65, 200, 1000])
@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
def test_route_tokens(T, bf16):
    check_route(logits_for(T, 128, 1, bf16), bf16)


@pytest.mark.parametrize("E,topk", [(1, 1), (2, 2), (8, 2), (60, 4), (63, 1), (64, 8), (65, 9), (128, 8), (160, 6), (256, 8),
                                    (257, 32), (384, 6), (512, 10), (1000, 8), (1024, 32)])
@pytest.mark.parametrize("score", [SOFT, SIG], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("steered", [False, True], ids=["plain", "bias"])
def test_route_experts(E, topk, score, steered):
    bias = np.random.default_rng(E).normal(0, 0.05, E).astype(np.float32) if steered else None
    for T, masked, renorm in ((37, 0.0, 1), (90, 0.3, 0)):
        check_route(logits_for(T, E, 2, False, masked), bias=bias, topk=topk, score=score, renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("E,groups,kept", [(8, 4, 2), (64, 8, 3), (64, 64, 5), (72, 8, 4), (160, 8, 3), (256, 8, 4),
                                           (320, 8, 7), (1024, 32, 4), (96, 3, 1), (64, 2, 2)])
@pytest.mark.parametrize("top2", [0, 1], ids=["max", "top2"])
@pytest.mark.parametrize("steered", [False, True], ids=["plain", "bias"])
def test_route_groups(E, groups, kept, top2, steered):
    bias = np.random.default_rng(E).normal(0, 0.05, E).astype(np.float32) if steered else None
    for score, T, masked in ((SIG, 33, 0.0), (SOFT, 70, 0.5), (SIG, 5, 0.95)):
        check_route(logits_for(T, E, 3, True, masked), True, bias, topk=min(6, E), score=score, groups=groups,
                    topk_groups=kept, group_score=top2)


@pytest.mark.parametrize("score", [SOFT, SIG], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("steered", [False, True], ids=["plain", "bias"])
def test_route_masks_and_extremes(score, steered):
    E = 70
    low_f32, low_bf16 = np.float32(-orows.FLT_MAX), wl.bf16_bits_to_f32(np.array([0xFF7F], dtype=np.uint16))[0]
    for bf16, low in ((False, low_f32), (True, low_bf16)):
        l = logits_for(80, E, 4, bf16)
        l[0] = -INF                                  # nothing open
        l[1] = NAN
        l[2], l[2, 69] = -INF, 1.0                   # one expert open
        l[3] = low                                   # a mask of the type's lowest value everywhere
        l[4], l[4, 3:6] = low, 0.0                   # ... and nearly everywhere
        l[5, ::2] = NAN
        l[6, 10] = INF
        l[7], l[7, 64] = -200.0, 200.0               # exponentials out of range
        l[8] = 0.0                                   # all tied
        l[9, ::2], l[9, 1::2] = 0.0, -0.0            # the same number
        l[10:20] = np.round(l[10:20] * 2) / 2        # many ties
        l[79] = -INF
        bias = None
        if steered:
            bias = np.round(np.random.default_rng(1).normal(0, 0.1, E), 2).astype(np.float32)
            bias[5], bias[6], bias[7] = -INF, NAN, 1000.0
        for renorm in (0, 1):
            check_route(l, bf16, bias, score=score, renormalize=renorm)
            check_route(l, bf16, bias, score=score, renormalize=renorm, groups=7, topk_groups=3, group_score=int(steered))


@pytest.mark.parametrize("E,topk,groups,kept", [(384, 6, 1, 1), (512, 10, 8, 3), (160, 6, 8, 3), (128, 20, 1, 1)])
@pytest.mark.parametrize("T", [1025, 8192, 8209, 17001])
def test_route_prompts_of_a_wave_per_token(E, topk, groups, kept, T):
    """Prompts with more than 256 experts, groups that are not whole 16s, more than 16 choices: blocks of one and of
    several rounds of 16 tokens."""
    top2 = int(T % 2 == 1 and groups > 1)
    bias = np.round(np.random.default_rng(E).normal(0, 0.05, E), 3).astype(np.float32) if T == 8209 else None
    l = logits_for(T, E, 81, False, 0.2)
    l[T // 3], l[T - 1] = -INF, -INF
    check_route(l, bias=bias, topk=topk, score=SIG, groups=groups, topk_groups=kept, group_score=top2)


@pytest.mark.parametrize("E,groups", [(40, 1), (70, 1), (256, 8), (300, 1)])
@pytest.mark.parametrize("T", [5, 50])
@pytest.mark.parametrize("steered", [False, True], ids=["plain", "bias"])
def test_route_every_kind_of_nan(E, groups, T, steered):
    """NaN of both signs, quiet and signalling, smallest and largest payload, are closed: in logits of both types and biases."""
    kinds = np.array([0x7FC00000, 0xFFC00000, 0x7F800001, 0xFF800001, 0x7FFFFFFF, 0xFFFFFFFF, 0x7FA00000], dtype=np.uint32)
    kinds16 = np.array([0x7FC0, 0xFFC0, 0x7F81, 0xFF81, 0x7FFF, 0xFFFF, 0x7FA0], dtype=np.uint16)
    rng = np.random.default_rng([E, T])
    r = q.make_router(E, 6, SIG, groups, min(3, groups), q.QLIN_GROUP_TOP2)
    l = logits_for(T, E, 71, True)
    gone = rng.random((T, E)) < 0.3
    gone[T // 2] = True
    which = rng.integers(0, 7, (T, E))
    bias, bias_ref = None, None
    if steered:
        bias = rng.normal(0, 0.05, E).astype(np.float32)
        bias_ref = bias.copy()
        bias.view(np.uint32)[3:10], bias_ref[3:10] = kinds, NAN
    want = orows.route(np.where(gone, NAN, l), 6, SIG, bias_ref, groups, min(3, groups), 1)
    wide = np.where(gone, kinds[which], l.view(np.uint32)).astype(np.uint32)
    half = np.where(gone, kinds16[which], to_bits(l)).astype(np.uint16)
    for logits, lt in ((to_dev(wide.view(np.int32)), F32), (to_dev_bf16(half), BF16)):
        got = run_route(r, logits, T, E, lt, bias)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[3], want[3]) and np.array_equal(got[4], want[4])
        assert np.isfinite(got[1]).all()


def test_route_strided_logits_and_sub_byte_alignment():
    check_route(logits_for(50, 60, 5, False), ld=61)
    check_route(logits_for(50, 60, 5, True), True, ld=61)
    l = logits_for(20, 60, 5, True)
    buf = torch.zeros(20 * 61 + 1, dtype=torch.int16, device=DEV)
    buf[1:].view(20, 61)[:, :60] = to_dev_bf16(to_bits(l))
    got = run_route(q.make_router(60, 4), buf[1:], 20, 61, BF16, None)
    assert np.array_equal(got[0], orows.route(l, 4)[0])


def test_route_many_tokens():
    """More tokens than 512 blocks of 16, and one expert that takes them all."""
    l = logits_for(20011, 8, 6, False)
    l[:, 3] += 50.0
    got = check_route(l, topk=2)
    assert got[2][4] - got[2][3] == 20011


@pytest.mark.parametrize("E,groups,kept", [(40, 1, 1), (64, 4, 2), (96, 6, 4), (128, 1, 1), (160, 10, 3), (200, 1, 1),
                                           (256, 8, 4), (256, 16, 5), (256, 1, 1), (72, 8, 4)])
@pytest.mark.parametrize("score", [SOFT, SIG], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("steered", [False, True], ids=["plain", "bias"])
def test_route_prompts(E, groups, kept, score, steered):
    """Prompts of over a thousand tokens, bf16 ties, masked experts, tokens with nothing open."""
    bias = np.round(np.random.default_rng(E).normal(0, 0.05, E), 3).astype(np.float32) if steered else None
    for T, bf16, masked, top2 in ((1029, True, 0.2, 1), (1500, False, 0.9, 0)):
        l = logits_for(T, E, 31, bf16, masked)
        l[T // 3], l[T - 1], l[5, ::2] = -INF, -INF, NAN
        if steered:
            bias[3], bias[E - 1] = -INF, NAN
        check_route(l, bf16, bias, topk=7, score=score, groups=groups, topk_groups=kept, group_score=top2,
                    renormalize=1 - top2)


@pytest.mark.parametrize("E,groups,kept", [(48, 3, 2), (60, 1, 1), (128, 8, 4), (128, 1, 1), (256, 8, 4), (250, 1, 1)])
@pytest.mark.parametrize("steered", [False, True], ids=["plain", "bias"])
def test_route_around_the_block_sizes(E, groups, kept, steered):
    """Around the token counts where the blocks of tokens change."""
    bias = np.random.default_rng(E).normal(0, 0.05, E).astype(np.float32) if steered else None
    for T in (31, 32, 33, 47, 48, 49, 63, 66, 4095, 4096, 4097, 6001):
        l = logits_for(T, E, 41, False, 0.1)
        l[T - 1], l[T // 2, ::3] = -INF, NAN
        check_route(l, bias=bias, topk=5, score=SIG, groups=groups, topk_groups=kept, group_score=int(steered))


@pytest.mark.parametrize("E", [60, 65, 128, 160, 256, 300])
@pytest.mark.parametrize("steered", [False, True], ids=["plain", "bias"])
def test_route_few_tokens(E, steered):
    bias = np.random.default_rng(E).normal(0, 0.05, E).astype(np.float32) if steered else None
    for T in (1, 2, 7, 8, 9, 16, 17):
        l = logits_for(T, E, 51, True, 0.2)
        l[T // 2, 1::2] = -INF
        check_route(l, True, bias, topk=9, score=SIG)
        check_route(l, True, bias, topk=3, renormalize=0)


@pytest.mark.parametrize("E", [24, 70, 128, 300])
@pytest.mark.parametrize("T", [3, 40, 90])
@pytest.mark.parametrize("steered", [False, True], ids=["plain", "bias"])
def test_route_sigmoid_of_low_logits(E, T, steered):
    """Sigmoids far below what 32 bits hold still have a ratio: the renormalized weights are that."""
    rng = np.random.default_rng([E, T])
    bias = np.round(rng.normal(0, 0.05, E), 2).astype(np.float32) if steered else None
    low = np.array([-80.0, -86.0, -90.0, -103.0, -120.0, -300.0, -700.0, -2000.0, 3.0])
    for first in range(0, len(low), 3):      # few tokens see every level too
        l = (low[(np.arange(T) + first) % len(low), None] - rng.uniform(0.0, 4.0, (T, E))).astype(np.float32)
        l[0] = -INF
        l[0, [3, 9]] = -100.0, -101.0
        l[1, ::2] -= 5.0
        l[2] = rng.uniform(-720.0, -700.0, E)    # on both sides of what is 0 in 64 bits, too
        l[2, 5:8] = -709.7826, -709.7828, -710.0
        for renorm in (1, 0):
            check_route(l, bias=bias, topk=min(E, 8), score=SIG, renormalize=renorm, scale=2.5)
            check_route(wl.bf16_bits_to_f32(to_bits(l)), True, bias, topk=3, score=SIG, renormalize=renorm)


@pytest.mark.parametrize("E,groups", [(256, 8), (300, 1), (64, 1)])
def test_route_one_workspace_for_all_sizes(E, groups):
    """A workspace of the largest call's size serves the smaller ones."""
    r = q.make_router(E, 4, SIG, groups, min(4, groups))
    sizes = (5000, 4096, 300, 33, 9, 1)
    work = guarded((q.qlin_route_workspace_bytes(r, max(sizes)),), torch.uint8, 0xEE)
    for T in sizes:
        l = logits_for(T, E, 61, False)
        bufs = [guarded(s, d, -7) for s, d in (((T, 4), torch.int32), ((T, 4), torch.float32), ((E + 1,), torch.int32),
                                               ((T * 4,), torch.int32), ((T, 4), torch.int32))]
        q.qlin_route(r, T, to_dev(l), E, F32, None, *bufs, work)
        torch.cuda.synchronize()
        check_guards(*bufs, work, what=f"qlin_route T={T}")
        want = orows.route(l, 4, SIG, None, groups, min(4, groups))
        for i, j in ((0, 0), (2, 2), (3, 3), (4, 4)):
            assert np.array_equal(bufs[i].cpu().numpy(), want[j])


@pytest.mark.parametrize("E", [65, 100, 128, 200, 256])
@pytest.mark.parametrize("score", [SOFT, SIG], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("spread", [1e-16, 4e-16, 3e-15, 1e-8, 1.0])
def test_route_same_choice_in_calls_of_any_size(E, score, spread):
    """Scores a few units in the last of 64 bits apart, or ordinary ones: a token chooses the same experts in a call of
    8 tokens (a wave each), of 40 and of 2000 (16 lanes each)."""
    T = 2000
    rng = np.random.default_rng([E, score])
    l = (rng.normal(size=(T, E)) * spread).astype(np.float32)
    l[rng.random((T, E)) < 0.1] = -INF
    for bias in (np.zeros(E), rng.choice([0.0, 0.25], E), rng.normal(0, 0.1, E)):
        router, ids = q.make_router(E, 7, score), {}
        ld, bd = to_dev(l), to_dev(bias.astype(np.float32))
        work = torch.empty(max(16, q.qlin_route_workspace_bytes(router, T)), dtype=torch.uint8, device=DEV)
        for n in (8, 40, T):
            got = torch.empty(T, 7, dtype=torch.int32, device=DEV)
            w, slots = torch.empty(n, 7, device=DEV), torch.empty(n, 7, dtype=torch.int32, device=DEV)
            off, rows = torch.empty(E + 1, dtype=torch.int32, device=DEV), torch.empty(n * 7, dtype=torch.int32, device=DEV)
            for t in range(0, T, n):
                q.qlin_route(router, n, ld[t:], E, F32, bd, got[t:], w, off, rows, slots, work)
            torch.cuda.synchronize()
            ids[n] = got.cpu().numpy()
        assert np.array_equal(ids[8], ids[40]) and np.array_equal(ids[8], ids[T])


def test_route_no_tokens():
    off = guarded((65,), torch.int32, -7)
    other = guarded((16,), torch.int32, -7)
    q.qlin_route(q.make_router(64, 8), 0, other, 64, F32, None, other, other, off, other, other)
    torch.cuda.synchronize()
    check_guards(off, other)
    assert int(off.abs().sum()) == 0 and int((other != -7).sum()) == 0


@pytest.mark.parametrize("T", [9, 300])
def test_route_on_another_stream_and_in_a_graph(T):
    """Replays follow new logits; eager work runs in between."""
    E, k = 128, 8
    router = q.make_router(E, k, SIG, 4, 2, q.QLIN_GROUP_TOP2)
    ls = [logits_for(T, E, s, False) for s in (21, 22, 23)]
    want = [orows.route(l, k, SIG, None, 4, 2, 1) for l in ls]
    stream = torch.cuda.Stream()
    ld = torch.empty(T, E, device=DEV)
    bufs = [torch.empty(n, dtype=d, device=DEV) for n, d in
            ((T * k, torch.int32), (T * k, torch.float32), (E + 1, torch.int32), (T * k, torch.int32), (T * k, torch.int32))]
    work = torch.empty(max(16, q.qlin_route_workspace_bytes(router, T)), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graph = None
    for i in (0, 1, 2, 0, 1):
        for b in bufs:
            b.fill_(-9)
        ld.copy_(to_dev(ls[i]))
        torch.cuda.synchronize()
        if graph is None:
            q.qlin_graph_begin(stream)
            q.qlin_route(router, T, ld, E, F32, None, *bufs, work, stream=stream)
            graph = q.qlin_graph_end(stream)
        q.qlin_graph_launch(graph, stream)
        torch.cuda.synchronize()
        got = [b.cpu().numpy() for b in bufs]
        assert np.array_equal(got[0].reshape(T, k), want[i][0]) and np.array_equal(got[2], want[i][2])
        assert np.array_equal(got[3], want[i][3]) and np.array_equal(got[4].reshape(T, k), want[i][4])
    q.qlin_graph_destroy(graph)


# ------------------------------------------------------------------ dispatch

FMTS = [wl.FP8_DYNAMIC, wl.W8A8_INT8, wl.BLOCK_FP8]


@pytest.mark.parametrize("fmt", FMTS, ids=["fp8_dynamic", "w8a8_int8", "block_fp8"])
@pytest.mark.parametrize("T,topk,K,pad", [(1, 1, 128, 0), (1, 8, 2048, 8), (7, 3, 2176, 0), (33, 8, 768, 64),
                                          (5, 32, 640, 0), (3, 2, 4224, 8), (4, 2, 8320, 0), (300, 4, 256, 0)])
def test_dispatch(fmt, T, topk, K, pad):
    x = wl.activations(fmt, 4096, K, T)
    x[T // 2, :128] = 0                                  # a group of zeros (a whole row where K is 128)
    qa, sa = oracle.quant_act(fmt, x)
    rng = np.random.default_rng([3, T, topk, K])
    total = T * topk + 5                                 # rows that no slot names stay
    slots = rng.permutation(total)[:T * topk].reshape(T, topk).astype(np.int32)
    slots[rng.random((T, topk)) < 0.1] = -1
    if T > 1:
        slots[0, 0], slots[1, 0] = total, -(1 << 31)     # out of range: skipped
    wide = np.zeros((T, K + pad), dtype=np.uint16)
    wide[:, :K] = x
    xq = guarded((total, K), torch.uint8, 0x55)
    xs = guarded(q.scales_shape(fmt, total, K, False), torch.float32, -1.0)
    print(f"[dispatch] fmt={fmt} T={T} topk={topk} K={K}", flush=True)
    q.qlin_dispatch_quantize(fmt, T, topk, K, to_dev_bf16(wide), K + pad, to_dev(slots), total, xq, xs)
    torch.cuda.synchronize()
    check_guards(xq, xs, what="qlin_dispatch_quantize")
    want_q = np.full((total, K), 0x55, dtype=np.uint8)
    want_s = np.full(tuple(xs.shape), -1.0, dtype=np.float32)
    for t in range(T):
        for s in slots[t]:
            if 0 <= s < total:
                want_q[s], want_s[s] = qa[t].view(np.uint8), sa[t]
    assert np.array_equal(as_u8(xq), want_q), "codes differ"
    assert np.array_equal(xs.cpu().numpy().view(np.uint32), want_s.view(np.uint32)), "scales differ"


def test_dispatch_more_groups_than_a_launch_has_threads_for():
    """2^20 tokens of 257 groups (64 GiB of x): 16 threads for each group are more than 2^32."""
    T, K, fmt = 1 << 20, 32896, wl.BLOCK_FP8
    if torch.cuda.mem_get_info()[0] < (80 << 30):
        torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < (80 << 30):
        pytest.skip("no 80 GiB of free memory")
    part = (1 << 27) // (K // 128)                       # tokens of a launch
    tokens = np.array([0, 1, part - 1, part, part + 1, 2 * part - 1, 2 * part, T - 1])
    x = torch.empty(T * K, dtype=torch.int16, device=DEV)
    rows = wl.activations(fmt, 4096, K, len(tokens))
    slots = np.full(T, -1, dtype=np.int32)
    for i, t in enumerate(tokens):
        x[int(t) * K:(int(t) + 1) * K] = to_dev_bf16(rows[i])
        slots[t] = len(tokens) - 1 - i
    xq = guarded((len(tokens), K), torch.uint8, 0x55)
    xs = guarded((len(tokens), K // 128), torch.float32, -1.0)
    print(f"[dispatch] T={T} K={K}, {part} tokens a launch", flush=True)
    q.qlin_dispatch_quantize(fmt, T, 1, K, x, K, to_dev(slots), len(tokens), xq, xs)
    torch.cuda.synchronize()
    check_guards(xq, xs, what="qlin_dispatch_quantize")
    qa, sa = oracle.quant_act(fmt, rows)
    assert np.array_equal(as_u8(xq)[::-1], qa.view(np.uint8)) and np.array_equal(xs.cpu().numpy()[::-1], sa)
    del x
    torch.cuda.empty_cache()


# ------------------------------------------------------------------- combine

def bits_of(v):
    return wl._to_bf16_bits(v.astype(np.float32))


@pytest.mark.parametrize("h32", [False, True], ids=["h_bf16", "h_f32"])
@pytest.mark.parametrize("y32", [False, True], ids=["y_bf16", "y_f32"])
@pytest.mark.parametrize("T,topk,N,add", [(1, 1, 16, None), (1, 8, 2048, "new"), (19, 8, 2064, None), (6, 32, 304, "y"),
                                          (130, 3, 4112, "new"), (40, 5, 768, "y")])
def test_combine(h32, y32, T, topk, N, add):
    rng = np.random.default_rng([4, T, topk, N])
    total, ldh, ldy, lda = T * topk + 3, N + 16, N + 8, N + 24
    h = rng.normal(size=(total, ldh)).astype(np.float32)
    r = rng.normal(size=(T, ldy if add == "y" else lda)).astype(np.float32)
    h_dev = to_dev(h) if h32 else to_dev_bf16(bits_of(h))
    h = h if h32 else wl.bf16_bits_to_f32(bits_of(h))
    r_bits = bits_of(r)
    r_ref = r if y32 else wl.bf16_bits_to_f32(r_bits)
    slots = rng.permutation(total)[:T * topk].reshape(T, topk).astype(np.int32)
    w = rng.random((T, topk)).astype(np.float32)
    gone = rng.random((T, topk)) < 0.15
    slots[gone], w[gone] = rng.choice([-1, total, 1 << 30, -(1 << 31)], gone.sum()), NAN   # no such row: nothing is added
    if T > 3:
        slots[3], w[3] = -1, INF                                                  # a token without any row
    y = guarded((T, ldy), torch.float32 if y32 else torch.int16, 7)
    if add == "y":
        y.copy_(to_dev(r) if y32 else to_dev_bf16(r_bits))
    before = y.cpu().numpy().copy()
    a_dev = None if add is None else y if add == "y" else (to_dev(r) if y32 else to_dev_bf16(r_bits))
    print(f"[combine] h32={h32} y32={y32} T={T} topk={topk} N={N} add={add}", flush=True)
    q.qlin_combine(T, topk, N, h_dev, ldh, F32 if h32 else BF16, to_dev(slots), to_dev(w), total, a_dev,
                   ldy if add == "y" else lda, y, ldy, F32 if y32 else BF16)
    torch.cuda.synchronize()
    check_guards(y, what="qlin_combine")
    got = y.cpu().numpy()
    assert np.array_equal(got[:, N:], before[:, N:]), "columns past N changed"
    got = got[:, :N] if y32 else wl.bf16_bits_to_f32(got.view(np.uint16)[:, :N])
    ref, size = orows.combine(h[:, :N], slots, w, None if add is None else r_ref[:, :N])
    # topk fused products and one sum, each rounded once; then the rounding of y (bf16 has 8 significant bits:
    # half a unit in the last place is up to 2^-8 of the value)
    tol = (topk + 2) * U * size
    tol = tol + (0 if y32 else 2.0 ** -8 * (np.abs(ref) + tol)) + 1e-37
    assert (np.abs(got - ref) <= tol).all(), f"off by {np.abs(got - ref).max()}"


def test_combine_keeps_infinities_and_nan_in_their_rows():
    h = torch.ones(4, 32, device=DEV)
    h[1, 3], h[2, 5] = NAN, INF
    slots = to_dev(np.array([[0, 1], [2, 3], [0, 3]], dtype=np.int32))
    w = torch.ones(3, 2, device=DEV)
    y = torch.zeros(3, 32, dtype=torch.bfloat16, device=DEV)
    q.qlin_combine(3, 2, 32, h, 32, F32, slots, w, 4, None, 0, y, 32, BF16)
    torch.cuda.synchronize()
    y = y.float().cpu().numpy()
    assert np.isnan(y[0, 3]) and np.isposinf(y[1, 5])
    y[0, 3] = y[1, 5] = 2.0
    assert (y == 2.0).all()


def test_combine_more_tokens_than_a_grid_row():
    T, N = 70001, 32
    h = torch.arange(T, device=DEV, dtype=torch.float32)[:, None].expand(T, N).contiguous()
    slots = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=DEV)
    w = torch.full((T, 1), 2.0, device=DEV)
    y = torch.empty(T, N, device=DEV)
    q.qlin_combine(T, 1, N, h, N, F32, slots, w, T, h, N, y, N, F32)
    torch.cuda.synchronize()
    assert torch.equal(y, h.flip(0) * 2 + h)


def test_combine_rows_far_apart():
    """Row offsets past 2^32 bytes, in the rows read and the rows written."""
    N, ld = 32, (1 << 30) + 64
    h = torch.empty(3 * ld, dtype=torch.bfloat16, device=DEV)
    y = torch.empty(2 * ld + N, dtype=torch.bfloat16, device=DEV)
    for i in range(3):
        h[i * ld:i * ld + N] = float(i + 1)
    slots = to_dev(np.array([[2, 0], [1, 2], [0, 1]], dtype=np.int32))
    w = to_dev(np.array([[1.0, 0.5], [2.0, 1.0], [1.0, 1.0]], dtype=np.float32))
    q.qlin_combine(3, 2, N, h, ld, BF16, slots, w, 3, None, 0, y, ld, BF16)
    torch.cuda.synchronize()
    got = [y[i * ld:i * ld + N].float().cpu().numpy() for i in range(3)]
    assert (got[0] == 3.5).all() and (got[1] == 7.0).all() and (got[2] == 3.0).all()
