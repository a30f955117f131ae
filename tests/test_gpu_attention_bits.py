"""Probabilities of attention over the 8-bit cache have 16 bits of mantissa where y is
bf16 (24 where it is fp32), whatever their size, the scales of the pages beside theirs
and the number of rows that a sequence brings."""
import numpy as np
import pytest
import torch

import skinny_bit_gemm_amd as q
import workloads as wl
from oracle import attention as oa
from test_gpu_attention import BF16, F32, FP8, INT8, U, Call, scaled

pytestmark = pytest.mark.gpu

from _gpu import check_guards  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.lib()


def error_and_bound(c):
    """|y - oracle| and its bound.  E: the scores' errors, (D + 8) roundings of their terms, two of
    the exponent.  W: each p's terms leave 2^-16 of it (three terms: 2^-24), and it has up to 24
    roundings (its power of two, the page's scale, the joined waves and parts), 4 for each time the
    maximum moves (at most once for the 64 tokens of a step, and 40 times for scores in any order
    that fp32 powers tell apart), and one for each token that is added.  y: its sum and the
    quotient likewise, and half a step of bf16 at the largest value that y can have by then.
    Nothing depends on how small a probability is beside the largest, until p times the value is
    below 2^-126."""
    torch.cuda.synchronize()
    used, n = int(c.offsets[-1]), c.Hq * c.D
    full = c.y.cpu().numpy()[:used, :n]
    got = (full if c.out == F32 else wl.bf16_bits_to_f32(full.view(np.uint16))).reshape(used, c.Hq, c.D).astype(np.float64)
    y, W, E, _ = oa.attention(c.ref, c.offsets, c.lengths, c.table, c.q_np[:used], c.scale, bool(c.causal), c.window)
    adds = c.longest + 4 * min(40, c.longest // 64 + 1) + 24
    bound = E * U + W * ((2.0 ** -24 if c.out == F32 else 2.0 ** -16) + adds * U) + np.abs(y) * adds * U + 2.0 ** -126
    if c.out == BF16:
        bound = bound + np.exp2(np.floor(np.log2(np.abs(y) + bound)) - 8)
    return np.abs(got - y), bound


def check(c):
    c.run()
    err, bound = error_and_bound(c)
    check_guards(c.y, c.work, what="qlin_cache_attention")
    at = np.unravel_index(np.argmax(err / bound), err.shape)
    print(f"  worst {(err / bound)[at]:.3f} of the bound at {at}", flush=True)
    assert (err <= bound).all(), f"off by {(err / bound)[at]:.4g} bounds at {at}"


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("out", [BF16, F32])
def test_as_many_bits_with_many_rows_as_with_few(D, out):
    for fmt, new, lengths in ((FP8, [300, 20], [300, 330]), (INT8, [180], [180]), (FP8, [9, 1], [60, 300])):
        check(Call(fmt, new, lengths, 8, 2, D, 32, out, seed=1))


def one_large(c, fmt, drop):
    """The first token of a sequence gets nearly all the weight, and its value is 0; all others are
    2^-drop of it.  The last channel holds a page's maximum, the scale that the others are small beside."""
    one = 0x38 if fmt == FP8 else 1                                   # the code of 1
    for s in range(len(c.lengths)):
        for which in range(c.table.shape[1]):
            p = c.ref.page_of(c.table, s, which * c.ref.page)
            if p < 0:
                continue
            c.ref.scales[0][p] = 1.0
            keys, index = c.ref.codes[0][p], c.ref.index[0]
            keys[:] = 0
            if which == 0:
                keys[:, index[0, 0]] = one
                c.ref.codes[1][p][:, c.ref.index[1][0]] = 0
    c.scale = float(np.float32(np.log(2.0)))                                   # scores in powers of two
    c.attention = q.make_attention(c.Hq, c.scale, c.causal, c.window)
    c.q_np[:, :, 0] = drop
    full = np.zeros((max(1, c.T), c.ldq), np.float32)
    full[:, :c.Hq * c.D] = c.q_np.reshape(len(c.q_np), -1)
    c.q.copy_(torch.from_numpy(full).to(torch.bfloat16).view(c.q.dtype).to(c.q.device))
    c.arrays[0].copy_(torch.from_numpy(c.ref.codes[0]))
    c.arrays[1].copy_(torch.from_numpy(c.ref.codes[1]))
    c.arrays[2].copy_(torch.from_numpy(c.ref.scales[0]))


@pytest.mark.parametrize("drop", [10, 18, 21, 40])
@pytest.mark.parametrize("apart", [0, 5, 10])
def test_small_probabilities_beside_a_large_one(drop, apart):
    for fmt, new, lengths, D in ((FP8, [300, 1], [300, 200], 64), (INT8, [150], [400], 128), (FP8, [20], [1500], 64),
                                 (FP8, [1], [700], 128)):
        c = Call(fmt, new, lengths, 8, 1, D, 64, BF16, seed=2)
        one_large(c, fmt, drop)
        # the scale of a page is large for its last channel alone: there its other codes are 0
        scaled(c, 1, lambda w, s: 2.0 ** apart if w == 1 else 1.0)
        for s in range(len(lengths)):
            p = c.ref.page_of(c.table, s, c.ref.page)
            c.ref.codes[1][p][:, c.ref.index[1][:, :D - 1]] = 0
        c.arrays[1].copy_(torch.from_numpy(c.ref.codes[1]))
        check(c)


def test_many_small_probabilities_over_a_long_context():
    c = Call(FP8, [70], [9000], 4, 1, 64, 128, BF16, seed=3)
    one_large(c, FP8, 21)
    scaled(c, 1, lambda w, s: 2.0 ** 10 if w == 30 else 1.0)
    check(c)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("small,large", [(-60, 90), (-66, 85), (-20, 60)])
def test_rows_that_see_small_scales_alone(out, small, large):
    """A prompt's first rows see its first page only; a later page's scale is far larger."""
    for fmt, page in ((FP8, 16), (INT8, 64)):
        c = Call(fmt, [200, 90], [200, 90], 8, 2, 64, page, out, seed=4)
        scaled(c, 1, lambda w, s: 2.0 ** (small if w == 0 else large if w == 2 else 0))
        check(c)


@pytest.mark.parametrize("out", [BF16, F32])
def test_large_values(out):
    """Values whose magnitudes sum to nearly 2^119 over the tokens."""
    for fmt, new, lengths in ((FP8, [300], [400]), (INT8, [1, 2], [700, 30]), (FP8, [130, 1], [1500, 40])):
        c = Call(fmt, new, lengths, 8, 2, 64, 64, out, seed=5)
        most = max(np.abs(c.ref.exact(1, c.table, s, range(n))).sum(0).max() for s, n in enumerate(lengths))
        factor = 2.0 ** np.floor(119 - np.log2(most))
        assert factor * most < 2.0 ** 119
        scaled(c, 1, lambda w, s: factor)
        check(c)
