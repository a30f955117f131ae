"""The per-row calls refuse what they cannot take, before any HIP call (no
GPU: the addresses are never dereferenced)."""
import random

import pytest

import skinny_bit_gemm_amd as q

OK, EINVAL, EALIGN, ESHAPE, EWS = 0, 1, 2, 3, 4
A = 1 << 20
FP8, I8, BLK = q.QLIN_FP8_DYNAMIC, q.QLIN_W8A8_INT8, q.QLIN_BLOCK_FP8
BF16, F32, I32 = q.QLIN_OUT_BF16, q.QLIN_OUT_F32_ACC, q.QLIN_OUT_I32_ACC


def route(T=4, logits=A, ld=None, lt=F32, bias=None, ids=A, w=A, off=A, rows=A, slots=A, work=A, wsb=1 << 20, **r):
    router = q.make_router(**{"experts": 64, "topk": 8, **r})
    return q.qlin_route(router, T, logits, router.experts if ld is None else ld, lt, bias, ids, w, off, rows, slots,
                        work, wsb, stream=0, raise_on_error=False)


@pytest.mark.parametrize("bad", [
    dict(experts=0), dict(experts=1025), dict(topk=0), dict(topk=33), dict(experts=4, topk=5), dict(score=2),
    dict(groups=0), dict(groups=65, experts=65), dict(groups=3), dict(topk_groups=2), dict(groups=4, topk_groups=0),
    dict(groups=4, topk_groups=5), dict(group_score=2), dict(renormalize=2), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(logits=None), dict(ids=None), dict(w=None), dict(off=None), dict(rows=None),
    dict(slots=None), dict(lt=I32), dict(lt=9)])
def test_route_invalid_arguments(bad):
    assert route(**bad) == EINVAL


def test_route_other_refusals():
    assert q.qlin_route(None, 4, A, 64, F32, None, A, A, A, A, A, A, 1 << 20, stream=0, raise_on_error=False) == EINVAL
    assert route(T=-1) == ESHAPE
    assert route(T=(1 << 17) + 1) == ESHAPE           # T x topk over 2^20
    assert route(ld=63) == EALIGN
    assert route(logits=A + 2) == EALIGN
    assert route(logits=A + 1, lt=BF16) == EALIGN
    for name in ("ids", "w", "off", "rows", "slots", "bias"):
        assert route(**{name: A + 2}) == EALIGN
    r = q.make_router(64, 8)
    need = q.qlin_route_workspace_bytes(r, 4096)
    assert need > 0 and q.qlin_route_workspace_bytes(r, 1) == 0
    assert route(T=4096, work=None) == EWS
    assert route(T=4096, wsb=need - 1) == EWS
    assert route(T=4096, work=A + 8, wsb=need) == EALIGN
    with pytest.raises(q.QlinError):
        q.qlin_route_workspace_bytes(r, -1)
    with pytest.raises(q.QlinError):
        q.qlin_route_workspace_bytes(q.make_router(0, 1), 1)


def dispatch(fmt=FP8, T=4, topk=8, K=512, x=A, ldx=512, slots=A, total=32, xq=A, xs=A):
    return q.qlin_dispatch_quantize(fmt, T, topk, K, x, ldx, slots, total, xq, xs, stream=0, raise_on_error=False)


def test_dispatch_refusals():
    assert dispatch(fmt=7) == EINVAL
    for name in ("x", "slots", "xq", "xs"):
        assert dispatch(**{name: None}) == EINVAL
    for bad in (dict(T=-1), dict(topk=0), dict(topk=33), dict(T=1 << 18), dict(K=520), dict(K=0), dict(total=-1),
                dict(total=(1 << 20) + 1), dict(fmt=BLK, K=640 + 16)):
        assert dispatch(**{"ldx": 1 << 20, **bad}) == ESHAPE
    for bad in (dict(ldx=504), dict(ldx=516), dict(x=A + 8), dict(slots=A + 2), dict(xq=A + 8), dict(xs=A + 2)):
        assert dispatch(**bad) == EALIGN
    assert dispatch(T=0) == OK and dispatch(total=0) == OK      # nothing to store


def combine(T=4, topk=8, N=256, h=A, ldh=256, ht=BF16, slots=A, w=A, total=32, add=None, ldadd=0, y=A << 1, ldy=256,
            yt=BF16):
    return q.qlin_combine(T, topk, N, h, ldh, ht, slots, w, total, add, ldadd, y, ldy, yt, stream=0,
                          raise_on_error=False)


def test_combine_refusals():
    for bad in (dict(ht=I32), dict(yt=I32), dict(h=None), dict(slots=None), dict(w=None), dict(y=None),
                dict(add=A << 1, ldadd=264)):
        assert combine(**bad) == EINVAL
    for bad in (dict(T=-1), dict(topk=0), dict(topk=33), dict(T=1 << 18), dict(N=0), dict(N=248), dict(total=-1),
                dict(total=(1 << 20) + 1)):
        assert combine(**bad) == ESHAPE
    for bad in (dict(ldh=248), dict(ldh=260), dict(ldy=260), dict(ht=F32, ldh=258), dict(add=A, ldadd=248),
                dict(add=A + 8, ldadd=256), dict(h=A + 8), dict(y=A + 8), dict(slots=A + 2), dict(w=A + 2)):
        assert combine(**bad) == EALIGN
    assert combine(T=0) == OK


def lora(M=4, N=256, K=512, n=8, R=16, x=A, ldx=512, ids=A, a=A, b=A, ranks=None, scales=None, base=None, ldb=0,
         y=A << 1, ldy=256, out=BF16, work=A, wsb=1 << 30):
    return q.qlin_lora(M, N, K, n, R, x, ldx, ids, a, b, ranks, scales, base, ldb, y, ldy, out, work, wsb, stream=0,
                       raise_on_error=False)


def test_lora_refusals():
    for bad in (dict(out=I32), dict(x=None), dict(ids=None), dict(a=None), dict(b=None), dict(y=None),
                dict(base=A << 1, ldb=264)):
        assert lora(**bad) == EINVAL
    for bad in (dict(M=-1), dict(M=(1 << 20) + 1), dict(N=248), dict(N=0), dict(K=520), dict(K=0), dict(n=0),
                dict(n=4097), dict(R=0), dict(R=12), dict(R=264)):
        assert lora(**bad) == ESHAPE
    for bad in (dict(ldx=504), dict(ldx=516), dict(ldy=248), dict(ldy=260), dict(out=F32, ldy=258),
                dict(base=A, ldb=252), dict(x=A + 8), dict(ids=A + 2), dict(a=A + 8), dict(b=A + 8),
                dict(ranks=A + 2), dict(scales=A + 2), dict(base=A + 8, ldb=256), dict(y=A + 8), dict(work=A + 8)):
        assert lora(**bad) == EALIGN
    need = q.qlin_lora_workspace_bytes(4, 256, 512, 8, 16)
    assert lora(work=None) == EWS and lora(wsb=need - 1) == EWS
    assert lora(M=0, work=None) == OK and q.qlin_lora_workspace_bytes(0, 256, 512, 8, 16) == 0
    for bad in ((-1, 256, 512, 8, 16), (4, 248, 512, 8, 16), (4, 256, 512, 0, 16), (4, 256, 512, 8, 12)):
        with pytest.raises(q.QlinError):
            q.qlin_lora_workspace_bytes(*bad)


def counts_of_rows():
    """Every count around those where plans change, and random ones."""
    rng = random.Random(7)
    return sorted({max(0, c + d) for c in [1 << i for i in range(18)] + [48, 1024, 1536, 2400, 2500, 3750, 5000, 7500, 12288,
                                                                     15000, 16384 * 3] for d in range(-2, 3)} |
                  {rng.randint(0, 1 << 17) for _ in range(300)})


def test_an_adapter_workspace_for_the_most_rows_serves_fewer():
    for N, K, n, R in ((4096, 12288, 8, 64), (4096, 4096, 64, 64), (256, 512, 8, 16), (10240, 5120, 4096, 256),
                       (2048, 2048, 1, 8), (80, 96, 300, 24), (151936, 4096, 16, 32), (16, 1 << 20, 2, 40)):
        sizes = [q.qlin_lora_workspace_bytes(M, N, K, n, R) for M in counts_of_rows()]
        assert sizes == sorted(sizes), f"{N} x {K}, {n} of rank {R}"


def test_a_routing_workspace_for_the_most_tokens_serves_fewer():
    for E, k, groups in ((64, 8, 1), (60, 4, 1), (128, 8, 1), (256, 8, 8), (384, 6, 1), (160, 6, 8), (1024, 8, 1)):
        r = q.make_router(E, k, groups=groups, topk_groups=min(2, groups))
        sizes = [q.qlin_route_workspace_bytes(r, T) for T in counts_of_rows() if T * k <= 1 << 20]
        assert sizes == sorted(sizes), f"{E} experts in {groups} groups"
