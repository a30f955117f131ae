"""Norm and rotation of heads on the GPU against the 64-bit oracle, within the
rounding errors of fp32 sums and one final rounding."""
import numpy as np
import pytest
import torch

import skinny_bit_gemm_amd as q
import workloads as wl
from oracle import attention as oa

pytestmark = pytest.mark.gpu

from _gpu import check_guards, guarded, to_dev, to_dev_bf16  # noqa: E402

BF16, F32 = q.QLIN_OUT_BF16, q.QLIN_OUT_F32_ACC
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.lib()


def to_f32(a, f32):
    return a if f32 else wl.bf16_bits_to_f32(a.view(np.uint16))


def angles(positions, R, base=1e4):
    a = np.arange(positions)[:, None] * base ** (-np.arange(0, R, 2) / max(R, 1))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def check(T, Hq, Hk, D, R, inter=0, it=BF16, ot=BF16, norm="both", positions=50, in_place=False, amplitude=1.0, eps=1e-6,
          seed=0, stream=None):
    rng = np.random.default_rng([5, T, Hq, Hk, D, R, seed])
    pad = 16
    width = (Hq + 2 * Hk) * D + pad                      # a wider qkv row, and columns behind it
    x = (rng.normal(size=(T, width)) * amplitude).astype(np.float32)
    if T > 2:
        x[1, :D] = 0.0                                   # a head of zeros
    bits = x if it == F32 else wl._to_bf16_bits(x)
    x = bits if it == F32 else wl.bf16_bits_to_f32(bits)
    at = rng.integers(0, positions, T).astype(np.int32)
    if T > 4:
        at[2], at[3], at[4] = -1, positions, -(1 << 31)  # padding
    at[0] = positions - 1
    wq, wk = (1 + 0.3 * rng.normal(size=(2, D))).astype(np.float32)
    wq, wk = (wq if norm in ("both", "q") else None), (wk if norm in ("both", "k") else None)
    table = angles(positions, R)
    qkv = guarded((T, width), torch.float32 if it == F32 else torch.int16)
    qkv.copy_(to_dev(bits) if it == F32 else to_dev_bf16(bits))
    qv, kv = qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + Hk) * D]
    if in_place:
        qo, ko, ldqo, ldko = qv, kv, width, width
    else:
        kind = torch.float32 if ot == F32 else torch.int16
        qo, ko = guarded((T, Hq * D + pad), kind, 7), guarded((T, Hk * D + 2 * pad), kind, 7)
        ldqo, ldko = Hq * D + pad, Hk * D + 2 * pad
    print(f"[rope] T={T} Hq={Hq} Hk={Hk} D={D} R={R} inter={inter} {it}->{ot} norm={norm} in_place={in_place}", flush=True)
    rope = q.make_rope(Hq, Hk, D, R, positions, inter, eps)
    dev = lambda a: None if a is None else to_dev(a)  # noqa: E731
    q.qlin_norm_rope(rope, T, qv if Hq else None, width, kv if Hk else None, width, it, dev(wq), dev(wk),
                     dev(table) if R else None, to_dev(at), qo, ldqo, ko, ldko, ot, stream=stream)
    torch.cuda.synchronize()
    check_guards(qkv, qo, ko, what="qlin_norm_rope")
    for out, ld, H, col, w in ((qo, ldqo, Hq, 0, wq), (ko, ldko, Hk, Hq * D, wk)):
        if not H:
            continue
        full = out.cpu().numpy()
        got = to_f32(np.ascontiguousarray(full[:, :H * D]), ot == F32).reshape(T, H, D).astype(np.float64)
        src = x[:, col:col + H * D].reshape(T, H, D)
        ref, size = oa.norm_rope(src, w, eps, table, at, R, inter)
        live = (at >= 0) & (at < positions) if R else np.ones(T, bool)
        # the sum of D squares, its root, the quotient and the products: D / 2 + 10 roundings of the terms
        tol = size * (D / 2 + 10) * U + np.abs(ref) * (0 if ot == F32 else 2.0 ** -8) + 1e-37
        got_live, ref, tol = got[live], ref[live], tol[live]
        assert np.array_equal(np.isnan(got_live), np.isnan(ref))         # 0 / 0: a head of zeros with eps 0
        fine = ~np.isnan(ref)
        off = (np.abs(got_live - ref)[fine] / tol[fine]).max()
        assert off <= 1, f"off by {off} tolerances"
        before = src if in_place else np.full((T, H, D), 7 if ot == F32 else wl.bf16_bits_to_f32(np.array([7], np.uint16))[0])
        assert np.array_equal(got[~live], np.asarray(before, np.float64)[~live]), "padding rows changed"
        if not in_place:
            assert (full[:, H * D:] == 7).all(), "columns behind the heads changed"
    if in_place:
        kept = qkv.cpu().numpy()[:, (Hq + Hk) * D:]
        assert np.array_equal(kept.view(np.uint8), np.ascontiguousarray(bits[:, (Hq + Hk) * D:]).view(np.uint8).reshape(kept.view(np.uint8).shape))


@pytest.mark.parametrize("D,R", [(8, 8), (24, 16), (64, 64), (64, 32), (72, 40), (80, 80), (96, 48), (128, 128), (128, 64),
                                 (192, 192), (200, 104), (256, 256), (256, 64)])
@pytest.mark.parametrize("inter", [0, 1])
def test_widths(D, R, inter):
    check(7, 4, 2, D, R, inter)
    check(6, 3, 1, D, R, inter, F32, F32)


@pytest.mark.parametrize("it,ot", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
def test_types(it, ot):
    check(33, 16, 8, 128, 128, 0, it, ot)
    check(5, 5, 5, 64, 64, 1, it, ot)


@pytest.mark.parametrize("T,Hq,Hk", [(1, 16, 8), (1, 1, 1), (2, 64, 8), (61, 32, 4), (300, 7, 1), (1000, 64, 8), (1024, 9, 2), (1500, 3, 3), (5, 0, 3),
                                     (5, 9, 0), (2, 1024, 1024)])
def test_tokens_and_heads(T, Hq, Hk):
    check(T, Hq, Hk, 128, 128)


@pytest.mark.parametrize("norm", ["both", "q", "k", "none"])
@pytest.mark.parametrize("R", [0, 64])
def test_norms_and_no_rotation(norm, R):
    check(9, 6, 2, 64, R, norm=norm)


@pytest.mark.parametrize("it", [BF16, F32])
def test_in_place(it):
    check(70, 8, 4, 128, 128, 0, it, it, in_place=True)
    check(70, 8, 4, 128, 96, 1, it, it, in_place=True)
    check(1100, 2, 1, 64, 64, 0, it, it, in_place=True)


def test_amplitudes():
    for amplitude in (1e-12, 1e-4, 1e4, 1e12):
        check(6, 4, 2, 128, 128, amplitude=amplitude, eps=0.0 if amplitude > 1 else 1e-6)


def test_far_positions():
    check(40, 4, 2, 128, 128, positions=131072, it=F32, ot=F32)


def test_a_call_of_no_tokens_and_another_stream():
    r = q.make_rope(4, 2, 128, 128, 10)
    x = torch.zeros(4, 1024, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(10, 128, device="cuda")
    q.qlin_norm_rope(r, 0, x, 1024, x[:, 512:], 1024, BF16, None, None, t, torch.zeros(4, dtype=torch.int32, device="cuda"),
                     x, 1024, x[:, 512:], 1024)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    check(64, 8, 2, 128, 128, stream=s)
