"""The calls around an 8-bit cache refuse what they cannot take, before any HIP
call (no GPU: the addresses are never dereferenced)."""
import random

import pytest

import skinny_bit_gemm_amd as q

OK, EINVAL, EALIGN, ESHAPE, EWS = 0, 1, 2, 3, 4
A = 1 << 20
FP8, I8, BLK = q.QLIN_FP8_DYNAMIC, q.QLIN_W8A8_INT8, q.QLIN_BLOCK_FP8
BF16, F32, I32 = q.QLIN_OUT_BF16, q.QLIN_OUT_F32_ACC, q.QLIN_OUT_I32_ACC


def rope(T=4, x=A, ldq=1024, k=A, ldk=256, it=BF16, qn=A, kn=A, cs=A, at=A, qo=A << 1, ldqo=1024, ko=A << 1, ldko=256,
         ot=BF16, **r):
    r = q.make_rope(**{"q_heads": 8, "kv_heads": 2, "head_dim": 128, "rotary_dim": 128, "positions": 100, **r})
    return q.qlin_norm_rope(r, T, x, ldq, k, ldk, it, qn, kn, cs, at, qo, ldqo, ko, ldko, ot, stream=0,
                            raise_on_error=False)


@pytest.mark.parametrize("bad", [
    dict(q_heads=-1), dict(q_heads=1025), dict(kv_heads=-1), dict(kv_heads=1025), dict(q_heads=0, kv_heads=0),
    dict(head_dim=0), dict(head_dim=4), dict(head_dim=100), dict(head_dim=264), dict(rotary_dim=-8), dict(rotary_dim=136),
    dict(rotary_dim=20), dict(interleaved=2), dict(positions=0), dict(eps=-1e-6), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(it=I32), dict(ot=I32), dict(x=None), dict(k=None), dict(qo=None), dict(ko=None),
    dict(cs=None), dict(at=None), dict(qo=A, ot=F32), dict(ko=A, ldko=264), dict(qo=A, ldqo=1032)])
def test_rope_invalid_arguments(bad):
    assert rope(**bad) == EINVAL


def test_rope_other_refusals():
    assert q.qlin_norm_rope(None, 1, A, 1024, A, 256, BF16, A, A, A, A, A, 1024, A, 256, BF16, stream=0,
                            raise_on_error=False) == EINVAL
    assert rope(T=-1) == ESHAPE and rope(T=(1 << 20) + 1) == ESHAPE
    for bad in (dict(ldq=1016), dict(ldq=1028), dict(ldk=248), dict(ldqo=1016), dict(ldko=260), dict(it=F32, ldq=1026),
                dict(x=A + 8), dict(k=A + 8), dict(qo=A + 8), dict(ko=A + 8), dict(qn=A + 8), dict(kn=A + 4), dict(cs=A + 8),
                dict(at=A + 2)):
        assert rope(**bad) == EALIGN
    assert rope(T=0) == OK and rope(T=0, qn=None, kn=None) == OK
    # what a call does not use is not looked at
    assert rope(T=0, rotary_dim=0, positions=0, cs=None, at=None) == OK
    assert rope(T=0, kv_heads=0, k=None, ko=None, ldk=1, ldko=3) == OK
    assert rope(T=0, q_heads=0, x=None, qo=None, ldq=1, ldqo=3) == OK


def cache(fmt=FP8, heads=2, D=128, page=32, pages=10, kc=A, vc=A, ks=A, vs=A):
    return q.make_cache(fmt, heads, D, page, pages, kc, vc, ks, vs)


def sequences(B=3, T=4, width=5, context=100, offsets=A, lengths=A, table=A):
    return q.make_sequences(B, T, offsets, lengths, table, width, context)


BAD_CACHES = [(EINVAL, bad) for bad in (
    dict(fmt=BLK), dict(fmt=7), dict(fmt=-1), dict(heads=0), dict(heads=1025), dict(D=0), dict(D=80), dict(D=96), dict(D=320),
    dict(page=0), dict(page=8), dict(page=48), dict(page=256))] + [(ESHAPE, dict(pages=0)), (ESHAPE, dict(pages=(1 << 24) + 1))]
BAD_CACHE_ARRAYS = [(EINVAL, {n: None}) for n in ("kc", "vc", "ks", "vs")] + \
    [(EALIGN, dict(kc=A + 8)), (EALIGN, dict(vc=A + 4)), (EALIGN, dict(ks=A + 2)), (EALIGN, dict(vs=A + 1))]
BAD_COUNTS = [(ESHAPE, bad) for bad in (
    dict(B=-1), dict(B=(1 << 20) + 1), dict(T=-1), dict(T=(1 << 20) + 1), dict(width=0), dict(width=(1 << 24) + 1),
    dict(context=0), dict(context=(1 << 30) + 1))]
BAD_ARRAYS = [(EINVAL, {n: None}) for n in ("offsets", "lengths", "table")] + \
    [(EALIGN, {n: A + 2}) for n in ("offsets", "lengths", "table")]


def append(c=None, s=None, k=A, ldk=256, v=A, ldv=256, t=BF16):
    return q.qlin_cache_append(cache() if c is None else c, sequences() if s is None else s, k, ldk, v, ldv, t, stream=0,
                               raise_on_error=False)


def read(c=None, s=None, k=A, ldk=256, v=A, ldv=256, t=BF16):
    return q.qlin_cache_read(cache() if c is None else c, sequences() if s is None else s, k, ldk, v, ldv, t, stream=0,
                             raise_on_error=False)


def attend(c=None, s=None, x=A, ldq=1024, y=A << 1, ldy=1024, t=BF16, work=A, wsb=1 << 40, **a):
    a = q.make_attention(**{"q_heads": 8, "scale": 0.1, **a})
    return q.qlin_cache_attention(a, cache() if c is None else c, sequences() if s is None else s, x, ldq, y, ldy, t, work,
                                  wsb, stream=0, raise_on_error=False)


@pytest.mark.parametrize("call", [append, read, attend])
def test_caches_and_sequences_are_checked(call):
    for status, bad in BAD_CACHES + BAD_CACHE_ARRAYS:
        assert call(c=cache(**bad)) == status, bad
    for status, bad in BAD_COUNTS + BAD_ARRAYS:
        assert call(s=sequences(**bad)) == status, bad
    assert call(s=sequences(B=0)) == OK and call(s=sequences(T=0)) == OK
    name = {append: "qlin_cache_append", read: "qlin_cache_read", attend: "qlin_cache_attention"}[call]
    f, more = getattr(q, name), (A, 256, A, 256, BF16) if call is not attend else (A, 1024, A << 1, 1024, BF16, A, 1 << 30)
    first = (q.make_attention(8, 0.1),) if call is attend else ()
    assert f(*first, None, sequences(), *more, stream=0, raise_on_error=False) == EINVAL
    assert f(*first, cache(), None, *more, stream=0, raise_on_error=False) == EINVAL


def test_append_and_read_refusals():
    for call in (append, read):
        assert call(t=I32) == EINVAL
        for bad in (dict(ldk=248), dict(ldk=260), dict(ldv=248), dict(t=F32, ldv=258), dict(k=A + 8), dict(v=A + 8)):
            assert call(**bad) == EALIGN
    assert append(k=None) == EINVAL and append(v=None) == EINVAL and read(k=None, v=None) == EINVAL
    assert read(k=None, ldk=3, s=sequences(T=0)) == OK and read(v=None, ldv=3, s=sequences(T=0)) == OK


def test_cache_bytes():
    for fmt, H, D, page, pages in ((FP8, 8, 128, 64, 1000), (I8, 1, 256, 16, 1), (FP8, 1024, 192, 128, 1 << 24)):
        assert q.qlin_cache_bytes(q.make_cache(fmt, H, D, page, pages)) == (pages * H * page * D, pages * H * 4)
    for _, bad in BAD_CACHES:
        with pytest.raises(q.QlinError):
            q.qlin_cache_bytes(cache(**bad))


def test_attention_refusals():
    for bad in (dict(q_heads=0), dict(q_heads=7), dict(q_heads=1026), dict(causal=2), dict(window=-1),
                dict(scale=float("nan")), dict(scale=float("-inf")), dict(x=None), dict(y=None), dict(y=A), dict(t=I32)):
        assert attend(**bad) == EINVAL, bad
    for bad in (dict(ldq=1016), dict(ldq=1020), dict(ldy=1016), dict(t=F32, ldy=1026), dict(x=A + 8), dict(y=A + 8)):
        assert attend(**bad) == EALIGN, bad
    assert q.qlin_cache_attention(None, cache(), sequences(), A, 1024, A << 1, 1024, BF16, A, 1 << 30, stream=0,
                                  raise_on_error=False) == EINVAL
    long = sequences(B=1, T=1, context=100000, width=4000)
    need = q.qlin_cache_attention_workspace_bytes(q.make_attention(8, 0.1), cache(), long)
    assert need > 0
    assert attend(s=long, work=None) == EWS and attend(s=long, wsb=need - 1) == EWS and attend(s=long, work=A + 8) == EALIGN
    assert q.qlin_cache_attention_workspace_bytes(q.make_attention(8, 0.1), cache(), sequences(T=0)) == 0
    with pytest.raises(q.QlinError):
        q.qlin_cache_attention_workspace_bytes(q.make_attention(7, 0.1), cache(), sequences())


def test_a_workspace_for_the_most_serves_less():
    rng = random.Random(3)
    counts = sorted({max(0, (1 << i) + d) for i in range(15) for d in (-1, 0, 1)} | {rng.randint(1, 9000) for _ in range(40)})
    contexts = sorted({(1 << i) + d for i in range(1, 22) for d in (-1, 0, 1)} | {rng.randint(1, 1 << 20) for _ in range(40)})
    for heads, group, D in ((8, 8, 128), (8, 4, 64), (1, 1, 128), (1, 64, 256), (8, 2, 192), (3, 5, 128)):
        a, c = q.make_attention(heads * group, 0.1), q.make_cache(FP8, heads, D, 64, 10, A, A, A, A)
        size = lambda B, T, n: q.qlin_cache_attention_workspace_bytes(a, c, sequences(B=B, T=T, context=n))  # noqa: E731
        for _ in range(30):
            B, T, n = rng.choice(counts), rng.choice(counts), rng.choice(contexts)
            for grown in ([size(B, T, x) for x in contexts], [size(B, x, n) for x in counts], [size(x, T, n) for x in counts],
                          [size(x, x, n) for x in counts]):
                assert grown == sorted(grown), (heads, group, D, B, T, n)
