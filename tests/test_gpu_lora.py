"""Low-rank adapters on the GPU against the 64-bit oracle, within the
rounding errors that the two fp32-accumulated products can make."""
import numpy as np
import pytest
import torch

import skinny_bit_gemm_amd as q
import workloads as wl
from oracle import rows as orows

pytestmark = pytest.mark.gpu

from _gpu import DEV, check_guards, guarded, to_dev, to_dev_bf16  # noqa: E402

BF16, F32 = q.QLIN_OUT_BF16, q.QLIN_OUT_F32_ACC
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.lib()


def make(M, N, K, n, R, seed, used="mixed"):
    """x, A, B as bf16 bits, ids, ranks, scales.  What lies past an adapter's
    rank is NaN in A and B."""
    rng = np.random.default_rng([17, M, N, K, n, R, seed])
    x = wl._to_bf16_bits(rng.normal(size=(M, K)).astype(np.float32))
    A = wl._to_bf16_bits((rng.normal(size=(n, R, K)) * K ** -0.5).astype(np.float32))
    B = wl._to_bf16_bits((rng.normal(size=(n, N, R)) * R ** -0.5).astype(np.float32))
    ranks = rng.choice([R, R, max(1, R // 2), max(1, R - 3), 1, 0], n).astype(np.int32)
    ranks[0] = R
    for a in range(n):
        A[a, ranks[a]:] = 0x7FC0
        B[a, :, ranks[a]:] = 0x7FC0
    scales = rng.uniform(0.25, 2.0, n).astype(np.float32)
    ids = {"mixed": rng.integers(-1, n + 1, M), "one": np.zeros(M, int), "runs": np.arange(M) * n // M,
           "none": np.full(M, -1)}[used].astype(np.int32)
    if used == "mixed" and M > 4:
        ids[1], ids[2], ids[3] = -1, 1 << 30, -(1 << 31)      # no adapter
    return x, A, B, ids, ranks, scales


def f32_of(bits):
    return wl.bf16_bits_to_f32(bits)


def check(M, N, K, n, R, seed=0, used="mixed", out=BF16, base="new", pad=0, use_ranks=True, use_scales=True, rows=None,
          stream=None):
    x, A, B, ids, ranks, scales = make(M, N, K, n, R, seed, used)
    if not use_ranks:
        A[A == 0x7FC0], B[B == 0x7FC0] = 0x3C00, 0x3C00
    f32 = out == F32
    rng = np.random.default_rng(seed + 99)
    ldx, ldy, ldb = K + pad, N + pad, N + (pad if base == "y" else 2 * pad)
    xw = np.full((M, ldx), 0x7FC0, dtype=np.uint16)
    xw[:, :K] = x
    b = rng.normal(size=(M, ldb)).astype(np.float32)
    b_dev = to_dev(b) if f32 else to_dev_bf16(wl._to_bf16_bits(b))
    b_ref = b if f32 else f32_of(wl._to_bf16_bits(b))
    y = guarded((M, ldy), torch.float32 if f32 else torch.int16, 7)
    if base == "y":
        y.copy_(b_dev)
    before = y.cpu().numpy().copy()
    nb = q.qlin_lora_workspace_bytes(M, N, K, n, R)
    work = guarded((nb,), torch.uint8, 0xFF)                   # NaN everywhere, as left by somebody else
    args = [to_dev_bf16(xw), to_dev(ids), to_dev_bf16(A), to_dev_bf16(B), to_dev(ranks) if use_ranks else None,
            to_dev(scales) if use_scales else None]
    print(f"[lora] M={M} N={N} K={K} n={n} R={R} used={used} out={out} base={base} pad={pad}", flush=True)
    q.qlin_lora(M, N, K, n, R, args[0], ldx, *args[1:], None if base is None else y if base == "y" else b_dev, ldb, y,
                ldy, out, work, stream=stream)
    torch.cuda.synchronize()
    check_guards(y, work, what="qlin_lora")
    got = y.cpu().numpy()
    assert np.array_equal(got[:, N:].view(np.uint8), before[:, N:].view(np.uint8)), "columns past N changed"
    got = got[:, :N] if f32 else f32_of(got.view(np.uint16)[:, :N])
    pick = np.arange(M) if rows is None else np.unique(np.concatenate([[0, M - 1], rng.integers(0, M, rows)]))
    ref, of_v, of_terms = orows.lora(f32_of(x[pick]), ids[pick], f32_of(A), f32_of(B), ranks if use_ranks else None,
                                     scales if use_scales else None, None if base is None else b_ref[pick, :N])
    # fp32 sums of K and of R terms: each rounding is at most U of a partial
    # sum; the errors of n of them add up like sqrt(n), with a factor of 4 for
    # the worst of all outputs.  v as two (three) bf16 numbers between the
    # products: each rounding leaves up to 2^-8 of what it rounds.  One rounding
    # of y (bf16 has 8 significant bits).
    tol = 4 * (np.sqrt(K) + np.sqrt(R) + 4) * U * of_terms + (4 * U if f32 else 2.0 ** -16) * of_v
    tol = tol + 2 * U * np.abs(ref)
    tol = tol + (0 if f32 else 2.0 ** -8 * (np.abs(ref) + tol)) + 1e-37
    err = np.abs(got[pick] - ref)
    assert np.isfinite(got).all(), "NaN or infinity in y"
    assert (err <= tol).all(), f"off by {(err / tol).max():.3g} of the tolerance"
    return y


@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M", [1, 2, 15, 17, 33, 64, 65, 130, 257])
@pytest.mark.parametrize("R", [8, 16, 64])
def test_rows_and_ranks(M, R, out):
    check(M, 272, 1040, 7, R, out=out, pad=8)


@pytest.mark.parametrize("R", [8, 24, 32, 40, 72, 96, 128, 136, 256])
@pytest.mark.parametrize("M", [5, 90])
def test_all_ranks(R, M):
    check(M, 144, 528, 4, R, out=F32, base="y", pad=8)
    check(M, 144, 528, 4, R, out=BF16, base=None)


@pytest.mark.parametrize("N,K", [(16, 16), (16, 48), (48, 32), (1040, 80), (80, 2064), (4096, 2048), (2048, 6144),
                                 (10240, 5120)])
@pytest.mark.parametrize("M", [1, 20, 100])
def test_sizes(N, K, M):
    check(M, N, K, 5, 16, pad=16, rows=12)


@pytest.mark.parametrize("used", ["one", "runs", "none"])
@pytest.mark.parametrize("base", [None, "new", "y"])
@pytest.mark.parametrize("M", [48, 70, 1100])
def test_row_orders_and_bases(M, used, base):
    check(M, 96, 160, 6, 16, used=used, base=base, pad=8, rows=40)
    check(M, 96, 160, 6, 16, used=used, base=base, out=F32, rows=40)


@pytest.mark.parametrize("R", [8, 32, 64, 128])
@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
def test_many_rows(R, out):
    check(1025, 592, 272, 9, R, out=out, rows=60, pad=8)
    check(2100, 80, 96, 3, R, out=out, used="runs", rows=60)


@pytest.mark.parametrize("R", [16, 24, 40, 72, 136, 256])
@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
def test_wide_tiles_at_odd_ranks(R, out):
    """64-row tiles whose ranks do not fill a stage, or fill several; a last stage and a tile that are not whole."""
    check(1024 + 37, 528, 144, 3, R, out=out, rows=40, pad=8, base="y")
    check(1100, 1296, 80, 2, R, out=out, used="one", rows=30, base=None)


@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 72, 136, 256])
@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
def test_prompts(R, out):
    """Enough rows for 64-row tiles at every rank: odd counts, runs, single rows, tiles that are not whole."""
    check(2400, 528, 144, 3, R, out=out, rows=40, pad=8, base="y")
    check(2400 + 37, 592, 272, 40, R, out=out, rows=60, pad=8)
    check(3001, 1296, 80, 9, R, out=out, used="runs", rows=30, base=None)


@pytest.mark.parametrize("R", [16, 24])
@pytest.mark.parametrize("M", [1535, 1536, 2399])
def test_rows_where_the_tiles_change(M, R):
    check(M, 272, 208, 5, R, rows=50, base="y")
    check(M, 272, 208, 700, R, out=F32, rows=50)


@pytest.mark.parametrize("R", [8, 32, 64, 80])
def test_prompts_with_many_adapters_and_bad_rows(R):
    check(2500, 32, 32, 4096, R, rows=80)
    M, N, K = 2500, 64, 96
    x, A, B, ids, ranks, scales = make(M, N, K, 3, R, 8, "one")
    ranks[0] = 1
    x[77, 5], x[78, 6] = 0x7F80, 0x7FC0
    y = torch.zeros(M, N, device=DEV)
    work = torch.empty(q.qlin_lora_workspace_bytes(M, N, K, 3, R), dtype=torch.uint8, device=DEV)
    q.qlin_lora(M, N, K, 3, R, to_dev_bf16(x), K, to_dev(ids), to_dev_bf16(A), to_dev_bf16(B), to_dev(ranks),
                to_dev(scales), None, 0, y, N, F32, work)
    torch.cuda.synchronize()
    got = y.cpu().numpy()
    sign = np.sign(f32_of(A[0, 0, 5:6])[0] * f32_of(B[0, :, 0]))
    assert np.array_equal(got[77], sign * np.inf) and np.isnan(got[78]).all()
    assert np.isfinite(np.delete(got, [77, 78], 0)).all()


WIDE = [(15001, 8), (7501, 16), (5003, 24), (3751, 32), (3001, 40), (2500, 64), (2501, 72), (2600, 136), (2750, 256)]


@pytest.mark.parametrize("M,R", WIDE)
@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
def test_wide_tiles(M, R, out):
    """Enough rows for 64-row tiles at each rank: ranks that do not fill a stage or fill several, tiles and stages
    that are not whole, every order of the rows and every base."""
    check(M, 144, 96, 3, R, out=out, rows=30, pad=8, base="y")
    check(M, 80, 48, 40, R, out=out, rows=30)
    check(M, 144, 80, 7, R, out=out, used="runs", rows=30, base=None)
    check(M, 48, 32, 2, R, out=out, used="one", rows=30, base="y")
    for base in (None, "new", "y"):
        check(M, 48, 32, 2, R, out=out, used="none", rows=30, base=base, pad=8)


@pytest.mark.parametrize("M,N,R,out", [(1279, 15648, 8, BF16), (1280, 15632, 8, BF16), (1290, 15520, 16, BF16),
                                       (1290, 7760, 24, F32), (2499, 208, 48, BF16), (2500, 208, 48, F32)])
def test_rows_where_tiles_become_wide(M, N, R, out):
    check(M, N, 64, 5, R, out=out, rows=20, base="y")
    check(M, N, 64, 700, R, out=out, rows=20)


@pytest.mark.parametrize("M,R", [(2500, 64), (15001, 8)])
@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
def test_bad_rows_in_wide_tiles(M, R, out):
    """A NaN and an infinity in x stay in their rows of a wide tile; with rank 1 the infinity reaches y as one."""
    N, K = 64, 96
    x, A, B, ids, ranks, scales = make(M, N, K, 3, R, 6, "one")
    ranks[0] = 1
    outs = []
    for bad in (False, True):
        if bad:
            x[1, 5], x[M - 2, 6] = 0x7F80, 0x7FC0
        y = torch.zeros(M, N, dtype=torch.float32 if out == F32 else torch.int16, device=DEV)
        work = torch.empty(q.qlin_lora_workspace_bytes(M, N, K, 3, R), dtype=torch.uint8, device=DEV)
        q.qlin_lora(M, N, K, 3, R, to_dev_bf16(x), K, to_dev(ids), to_dev_bf16(A), to_dev_bf16(B), to_dev(ranks),
                    to_dev(scales), None, 0, y, N, out, work)
        torch.cuda.synchronize()
        outs.append(y.cpu().numpy() if out == F32 else f32_of(y.cpu().numpy().view(np.uint16)))
    sign = np.sign(f32_of(A[0, 0, 5:6])[0] * f32_of(B[0, :, 0]))
    assert np.array_equal(outs[1][1], sign * np.inf) and np.isnan(outs[1][M - 2]).all()
    assert np.array_equal(np.delete(outs[0], [1, M - 2], 0), np.delete(outs[1], [1, M - 2], 0))


@pytest.mark.parametrize("M,R", [(2, 16), (16, 64), (64, 16), (2500, 64), (9000, 16), (15001, 8), (6000, 8)])
@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
def test_same_bits_on_every_path(M, R, out):
    """One launch, direct tiles, sorted tiles of both heights, and more rows than a sorting thread holds: a second call
    gives the same bits, and so do the same rows when the others have other adapters."""
    N, K, n = 144, 272, 5
    x, A, B, ids, ranks, scales = make(M, N, K, n, R, 8, "runs")
    dev = [to_dev_bf16(x), to_dev_bf16(A), to_dev_bf16(B), to_dev(ranks), to_dev(scales)]
    work = torch.empty(q.qlin_lora_workspace_bytes(M, N, K, n, R), dtype=torch.uint8, device=DEV)
    outs = []
    for turn in range(4):
        i = ids.copy()
        if turn == 2:
            i[1::2] = np.random.default_rng(1).integers(-1, n, len(i[1::2]))
        if turn == 3:
            i[1::2] = -1
        y = torch.zeros(M, N, dtype=torch.float32 if out == F32 else torch.int16, device=DEV)
        q.qlin_lora(M, N, K, n, R, dev[0], K, to_dev(i), dev[1], dev[2], dev[3], dev[4], None, 0, y, N, out, work)
        torch.cuda.synchronize()
        outs.append(y.cpu().numpy())
    assert np.array_equal(outs[0], outs[1])
    assert np.array_equal(outs[0][::2], outs[2][::2]) and np.array_equal(outs[0][::2], outs[3][::2])


def test_the_largest_row_count():
    """2^20 rows: more row tiles than a grid's y holds."""
    M, N, K, n, R = 1 << 20, 16, 16, 2, 8
    x = torch.ones(M, K, dtype=torch.bfloat16, device=DEV)
    A = torch.ones(n, R, K, dtype=torch.bfloat16, device=DEV)
    B = torch.ones(n, N, R, dtype=torch.bfloat16, device=DEV)
    B[1] = 2.0
    ids = torch.arange(M, dtype=torch.int32, device=DEV) % 3        # adapter 2: none
    y = torch.full((M, N), -1.0, device=DEV)
    work = torch.empty(q.qlin_lora_workspace_bytes(M, N, K, n, R), dtype=torch.uint8, device=DEV)
    q.qlin_lora(M, N, K, n, R, x, K, ids, A, B, None, None, None, 0, y, N, F32, work)
    torch.cuda.synchronize()
    want = torch.tensor([128.0, 256.0, 0.0], device=DEV)[ids.long()]
    assert (y == want[:, None]).all()


def test_more_rows_than_the_sort_holds():
    """Rows past the 4096 that the sorting workgroup keeps in registers."""
    for used in ("mixed", "runs"):
        check(9001, 48, 64, 37, 8, used=used, rows=120)
    check(5000, 32, 32, 4096, 16, rows=80, out=F32)


@pytest.mark.parametrize("M", [1, 3, 16])
@pytest.mark.parametrize("R", [8, 16, 24, 40, 64])
def test_few_rows_of_small_adapters(M, R):
    check(M, 528, 272, 3, R, out=F32, base="y", pad=8)
    check(M, 48, 1040, 5, R, used="one")
    check(M, 1040, 528, 4, R, base=None, use_scales=False)


def test_defaults_and_many_adapters():
    check(40, 64, 64, 3, 16, use_ranks=False)
    check(40, 64, 64, 3, 16, use_scales=False)
    check(90, 32, 32, 4096, 8)
    check(1500, 32, 32, 4096, 8, rows=80)
    check(1500, 32, 32, 1, 8, rows=80)


def test_ranks_out_of_range_are_clamped():
    M, N, K, n, R = 6, 32, 64, 3, 8
    x, A, B, _, _, _ = make(M, N, K, n, R, 3)
    A[A == 0x7FC0], B[B == 0x7FC0] = 0x3C00, 0x3C00
    ids = np.array([0, 1, 2, 0, 1, 2], dtype=np.int32)
    ranks = np.array([100, -5, 3], dtype=np.int32)
    y = guarded((M, N), torch.float32, 7)
    work = guarded((q.qlin_lora_workspace_bytes(M, N, K, n, R),), torch.uint8, 0xFF)
    q.qlin_lora(M, N, K, n, R, to_dev_bf16(x), K, to_dev(ids), to_dev_bf16(A), to_dev_bf16(B), to_dev(ranks), None, None,
                0, y, N, F32, work)
    torch.cuda.synchronize()
    check_guards(y, work)
    ref, _, of_terms = orows.lora(f32_of(x), ids, f32_of(A), f32_of(B), ranks)
    assert (np.abs(y.cpu().numpy() - ref) <= 64 * U * of_terms).all()
    assert (y[1] == 0).all() and (y[4] == 0).all()


def test_a_bad_row_stays_alone():
    """NaN and infinities in one row's x change that row alone."""
    for M in (40, 90):
        x, A, B, ids, ranks, scales = make(M, 64, 96, 3, 16, 5, "one")
        outs = []
        for bad in (False, True):
            xb = x.copy()
            if bad:
                xb[7, 5], xb[7, 6] = 0x7FC0, 0x7F80
            y = torch.zeros(M, 64, device=DEV)
            work = torch.empty(q.qlin_lora_workspace_bytes(M, 64, 96, 3, 16), dtype=torch.uint8, device=DEV)
            q.qlin_lora(M, 64, 96, 3, 16, to_dev_bf16(xb), 96, to_dev(ids), to_dev_bf16(A), to_dev_bf16(B), to_dev(ranks),
                        to_dev(scales), None, 0, y, 64, F32, work)
            torch.cuda.synchronize()
            outs.append(y.cpu().numpy())
        others = np.arange(M) != 7
        assert np.array_equal(outs[0][others], outs[1][others])
        assert np.isnan(outs[1][7]).all()


@pytest.mark.parametrize("M", [2, 40, 90, 1100])
@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
def test_an_infinite_row(M, out):
    """An infinity in x of a row with an adapter of rank 1 leaves nothing to cancel: y is infinite, signed by B's columns."""
    N, K, R = 64, 96, 16
    x, A, B, ids, ranks, scales = make(M, N, K, 3, R, 6, "one")
    ranks[0] = 1
    x[1, 5] = 0x7F80
    assert (A[0, 0, 5] & 0x7FFF) and (B[0, :, 0] & 0x7FFF).all()
    y = torch.zeros(M, N, dtype=torch.float32 if out == F32 else torch.int16, device=DEV)
    work = torch.empty(q.qlin_lora_workspace_bytes(M, N, K, 3, R), dtype=torch.uint8, device=DEV)
    q.qlin_lora(M, N, K, 3, R, to_dev_bf16(x), K, to_dev(ids), to_dev_bf16(A), to_dev_bf16(B), to_dev(ranks),
                to_dev(scales), None, 0, y, N, out, work)
    torch.cuda.synchronize()
    got = y.cpu().numpy() if out == F32 else f32_of(y.cpu().numpy().view(np.uint16))
    sign = np.sign(f32_of(A[0, 0, 5:6])[0] * f32_of(B[0, :, 0]))
    assert np.array_equal(got[1], sign * np.inf)
    assert np.isfinite(np.delete(got, 1, 0)).all()


@pytest.mark.parametrize("M", [33, 500])
def test_same_bits_again_and_for_any_neighbours(M):
    """A second call gives the same bits, and so do the same rows when the
    others have other adapters."""
    N, K, n, R = 208, 400, 5, 16
    x, A, B, ids, ranks, scales = make(M, N, K, n, R, 8, "runs")
    dev = [to_dev_bf16(x), to_dev_bf16(A), to_dev_bf16(B), to_dev(ranks), to_dev(scales)]
    work = torch.empty(q.qlin_lora_workspace_bytes(M, N, K, n, R), dtype=torch.uint8, device=DEV)
    outs = []
    for turn in range(3):
        i = ids.copy()
        if turn == 2:
            i[1::2] = np.random.default_rng(1).integers(-1, n, len(i[1::2]))
        y = torch.zeros(M, N, device=DEV)
        q.qlin_lora(M, N, K, n, R, dev[0], K, to_dev(i), dev[1], dev[2], dev[3], dev[4], None, 0, y, N, F32, work)
        torch.cuda.synchronize()
        outs.append(y.cpu().numpy())
    assert np.array_equal(outs[0], outs[1])
    assert np.array_equal(outs[0][::2], outs[2][::2])


@pytest.mark.parametrize("M", [1, 5, 16, 40, 90, 2500, 4100])
@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
def test_rows_without_an_adapter_stay_as_they_are(M, out):
    """In place, rows without an adapter and of rank 0 keep every bit: negative zeros and NaN payloads too."""
    N, K, R = 80, 96, 16
    x, A, B, ids, ranks, scales = make(M, N, K, 3, R, 9, "one")
    ranks[1] = 0
    ids[:] = np.arange(M) % 4 - 1                  # none, full rank, rank 0, some rank
    rng = np.random.default_rng(M)
    word, special = (np.uint16, [0x8000, 0x7F81, 0xFFC1, 0x8001]) if out == BF16 else (
        np.uint32, [0x80000000, 0x7F800001, 0xFFC00001, 0x80000001])
    before = rng.choice(np.array(special, dtype=word), (M, N))
    y = to_dev(before.view(np.int16 if out == BF16 else np.int32))
    work = torch.empty(q.qlin_lora_workspace_bytes(M, N, K, 3, R), dtype=torch.uint8, device=DEV)
    q.qlin_lora(M, N, K, 3, R, to_dev_bf16(x), K, to_dev(ids), to_dev_bf16(A), to_dev_bf16(B), to_dev(ranks),
                to_dev(scales), y, N, y, N, out, work)
    torch.cuda.synchronize()
    stay = (ids == -1) | (ids == 1)
    assert np.array_equal(y.cpu().numpy().view(word)[stay], before[stay])


@pytest.mark.parametrize("R", [8, 64])
def test_one_workspace_for_all_sizes(R):
    """A workspace of the largest call's size serves the smaller ones, whatever is left in it."""
    N, K, n = 48, 1040, 5
    sizes = (2600, 1530, 130, 65, 64, 40, 20, 1)
    work = guarded((q.qlin_lora_workspace_bytes(max(sizes), N, K, n, R),), torch.uint8, 0xFF)
    for M in sizes:
        x, A, B, ids, ranks, scales = make(M, N, K, n, R, 3)
        y = guarded((M, N), torch.float32, 7)
        q.qlin_lora(M, N, K, n, R, to_dev_bf16(x), K, to_dev(ids), to_dev_bf16(A), to_dev_bf16(B), to_dev(ranks),
                    to_dev(scales), None, 0, y, N, F32, work)
        torch.cuda.synchronize()
        check_guards(y, work, what=f"qlin_lora M={M}")
        pick = np.unique(np.linspace(0, M - 1, 40).astype(int))
        ref, _, of_terms = orows.lora(f32_of(x[pick]), ids[pick], f32_of(A), f32_of(B), ranks, scales)
        err = np.abs(y.cpu().numpy()[pick] - ref)
        assert (err <= 4 * (np.sqrt(K) + 8) * U * (of_terms + np.abs(ref)) + 1e-37).all()


@pytest.mark.parametrize("M,R", [(2, 16), (40, 16), (40, 128), (90, 64), (2500, 64), (2500, 136), (15001, 8)])
@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
def test_products_that_cancel(M, R, out):
    """A x has 24 bits and B takes the difference of two ranks that agree in their first 16: what is left is exact,
    on every path."""
    N, K = 48, 64
    rng = np.random.default_rng([M, R])
    a = 1.0 + (2 * rng.integers(0, 64, 3) + 1) / 128.0               # eight bits each
    A, B = np.zeros((1, R, K)), np.zeros((1, N, R))
    A[0, 0, :3], A[0, 1, :2] = a, a[:2]
    B[0, :, 0], B[0, :, 1] = 1.0, -1.0
    x = np.zeros((M, K))
    x[:, :3] = 1.0, 2.0 ** -8, 2.0 ** -16
    bits = [to_dev_bf16(wl._to_bf16_bits(v.astype(np.float32))) for v in (x, A, B)]
    y = torch.zeros(M, N, dtype=torch.float32 if out == F32 else torch.int16, device=DEV)
    work = torch.empty(q.qlin_lora_workspace_bytes(M, N, K, 1, R), dtype=torch.uint8, device=DEV)
    q.qlin_lora(M, N, K, 1, R, bits[0], K, torch.zeros(M, dtype=torch.int32, device=DEV), bits[1], bits[2], None, None,
                None, 0, y, N, out, work)
    torch.cuda.synchronize()
    got = y.cpu().numpy() if out == F32 else f32_of(y.cpu().numpy().view(np.uint16))
    assert (got == np.float32(a[2] * 2.0 ** -16)).all()


def test_slices_of_a_wider_projection():
    """q, k, v: adapters for column ranges of one output, in place."""
    M, K, n, R, widths = 21, 256, 4, 16, (128, 64, 64)
    total = sum(widths)
    y = guarded((M, total), torch.float32, 0.0)
    base = np.random.default_rng(2).normal(size=(M, total)).astype(np.float32)
    y.copy_(to_dev(base))
    at = 0
    for i, N in enumerate(widths):
        x, A, B, ids, ranks, scales = make(M, N, K, n, R, 20 + i)
        work = torch.empty(q.qlin_lora_workspace_bytes(M, N, K, n, R), dtype=torch.uint8, device=DEV)
        view = y[:, at:at + N]
        q.qlin_lora(M, N, K, n, R, to_dev_bf16(x), K, to_dev(ids), to_dev_bf16(A), to_dev_bf16(B), to_dev(ranks),
                    to_dev(scales), view, total, view, total, F32, work)
        ref, _, of_terms = orows.lora(f32_of(x), ids, f32_of(A), f32_of(B), ranks, scales, base[:, at:at + N])
        torch.cuda.synchronize()
        err = np.abs(view.cpu().numpy() - ref)
        assert (err <= 4 * (np.sqrt(K) + 8) * U * (of_terms + np.abs(ref)) + 1e-37).all()
        at += N
    check_guards(y)


def test_rows_and_adapters_far_apart():
    """Offsets past 2^32 bytes: an adapter far into A, rows far apart in x and y."""
    N, K, n, R = 32, 32768, 300, 256
    ld = (1 << 30) + 64
    A = torch.zeros(n * R * K, dtype=torch.bfloat16, device=DEV)            # 5 GB
    B = torch.zeros(n, N, R, dtype=torch.bfloat16, device=DEV)
    A.view(n, R, K)[n - 1, 3, :] = 0.5
    B[n - 1, :, 3] = 2.0
    for M in (3, 70):
        x = torch.ones((M, K), dtype=torch.bfloat16, device=DEV)
        ids = torch.full((M,), n - 1, dtype=torch.int32, device=DEV)
        y = torch.zeros(M, N, device=DEV)
        work = torch.empty(q.qlin_lora_workspace_bytes(M, N, K, n, R), dtype=torch.uint8, device=DEV)
        q.qlin_lora(M, N, K, n, R, x, K, ids, A, B, None, None, None, 0, y, N, F32, work)
        torch.cuda.synchronize()
        assert (y == float(K)).all()
    del A
    xw = torch.empty(2 * ld + 64, dtype=torch.bfloat16, device=DEV)
    yw = torch.empty(2 * ld + N, dtype=torch.bfloat16, device=DEV)
    A2 = torch.ones(1, 8, 64, dtype=torch.bfloat16, device=DEV)
    B2 = torch.ones(1, N, 8, dtype=torch.bfloat16, device=DEV)
    for i in range(3):
        xw[i * ld:i * ld + 64] = float(i)
        yw[i * ld:i * ld + N] = 1.0
    ids = torch.zeros(3, dtype=torch.int32, device=DEV)
    work = torch.empty(q.qlin_lora_workspace_bytes(3, N, 64, 1, 8), dtype=torch.uint8, device=DEV)
    q.qlin_lora(3, N, 64, 1, 8, xw, ld, ids, A2, B2, None, None, yw, ld, yw, ld, BF16, work)
    torch.cuda.synchronize()
    for i in range(3):
        assert (yw[i * ld:i * ld + N].float() == torch.tensor(1.0 + 512.0 * i).bfloat16().float().item()).all()


@pytest.mark.parametrize("M", [12, 200])
def test_on_another_stream_and_in_a_graph(M):
    N, K, n, R = 144, 272, 4, 16
    x, A, B, ids, ranks, scales = make(M, N, K, n, R, 12)
    order = [ids, np.roll(ids, 5), np.zeros_like(ids)]
    dev = [to_dev_bf16(x), to_dev_bf16(A), to_dev_bf16(B), to_dev(ranks), to_dev(scales)]
    idd, y = to_dev(ids), torch.empty(M, N, device=DEV)
    work = torch.empty(q.qlin_lora_workspace_bytes(M, N, K, n, R), dtype=torch.uint8, device=DEV)
    stream, graph = torch.cuda.Stream(), None
    torch.cuda.synchronize()
    for i in (0, 1, 2, 1, 0):
        idd.copy_(to_dev(order[i]))
        y.fill_(-5.0)
        torch.cuda.synchronize()
        if graph is None:
            q.qlin_graph_begin(stream)
            q.qlin_lora(M, N, K, n, R, dev[0], K, idd, dev[1], dev[2], dev[3], dev[4], None, 0, y, N, F32, work,
                        stream=stream)
            graph = q.qlin_graph_end(stream)
        q.qlin_graph_launch(graph, stream)
        torch.cuda.synchronize()
        ref, _, of_terms = orows.lora(f32_of(x), order[i], f32_of(A), f32_of(B), ranks, scales)
        assert (np.abs(y.cpu().numpy() - ref) <= 4 * (np.sqrt(K) + 8) * U * of_terms + 1e-37).all()
    q.qlin_graph_destroy(graph)
