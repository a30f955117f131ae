"""Attention over the 8-bit cache on the GPU against the 64-bit oracle, within
the rounding errors that fp32 scores, sums and the probabilities' terms can make.
What no token sees (behind a sequence's end, before its window, in absent pages)
holds NaN codes and scales."""
import numpy as np
import pytest
import torch

import skinny_bit_gemm_amd as q
import workloads as wl
from oracle import attention as oa

pytestmark = pytest.mark.gpu

from _gpu import check_guards, guarded, to_dev, to_dev_bf16  # noqa: E402

BF16, F32 = q.QLIN_OUT_BF16, q.QLIN_OUT_F32_ACC
FP8, INT8 = q.QLIN_FP8_DYNAMIC, q.QLIN_W8A8_INT8
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.lib()


def random_codes(rng, fmt, shape):
    if fmt == INT8:
        return rng.integers(-127, 128, shape).astype(np.int8).view(np.uint8)
    c = rng.integers(0, 0x7F, shape).astype(np.uint8)                # no NaN
    return np.where(c >= 0x60, c - 0x30, c).astype(np.uint8) | (rng.integers(0, 2, shape) << 7).astype(np.uint8)


def make_cache(rng, fmt, H, D, page, lengths, table, pages, low=None):
    """Random codes where tokens low[s] .. lengths[s] - 1 are, NaN elsewhere;
    pages' scales differ by up to 2^6."""
    c = oa.Cache(fmt, H, D, page, pages, 0x7F)
    for s, n in enumerate(lengths):
        for which in range(-(-min(max(int(n), 0), table.shape[1] * page) // page)):
            p = c.page_of(table, s, which * page)
            lo, hi = max(0, (0 if low is None else low[s]) - which * page), min(page, int(n) - which * page)
            if p < 0 or hi <= lo:
                continue
            for kv in range(2):
                top = 127.0 if fmt == INT8 else 16.0
                c.scales[kv][p] = (np.exp2(rng.uniform(-3, 3, H)) * (1.0 if kv else 0.7) / top).astype(np.float32)
                index = c.index[kv][lo:hi]
                c.codes[kv][p][:, index] = random_codes(rng, fmt, (H,) + index.shape)
    return c


def table_of(rng, lengths, page, pages, width=None):
    held = [-(-max(int(n), 0) // page) for n in lengths]
    table = np.full((len(lengths), width or max(held) + 1), -1, dtype=np.int32)
    free = rng.permutation(pages)[:sum(held)]
    for i, n in enumerate(held):
        table[i, :n], free = free[:n], free[n:]
    return table


def tolerance(y, W, E, F, D, longest, out, many):
    """E: the scores' errors, (D + 8) roundings of their terms, two of the exponent.
    W: each p has up to 8 roundings (its power of two, the page's scale, the joined
    waves and parts) and 4 for each time the maximum moves, at most once for the 64
    tokens of a step, and at most 40 times for scores in any order that fp32 powers
    tell apart; its terms leave 2^-16 (three terms, where y is fp32: 2^-24; one fp16
    number, where y is bf16 and the sequence has many rows: 2^-11 of a normal number,
    and 2^-25 below them, where scales are at least 2^-4: F 2^-21); the product's sum
    has a rounding for each of the longest / 4 tokens of a wave (each of all of them,
    where there are many rows).  y: the sum of p likewise, the quotient, and the
    rounding of y."""
    moves = 4 * min(40, longest // 64 + 1)
    many = np.asarray(many)[:, None, None]
    terms = 2.0 ** -24 if out == F32 else np.where(many, 2.0 ** -11, 2.0 ** -16)
    flat = 0.0 if out == F32 else np.where(many, 2.0 ** -21, 0.0)
    adds = longest * np.where(many, 1.0, 0.25)
    return E * U + W * (terms + (8 + moves + adds + 16) * U) + F * flat + np.abs(y) * (
        (adds + moves + 24) * U + (0 if out == F32 else 2.0 ** -8)) + 1e-30


class Call:
    def __init__(self, fmt, new, lengths, Hq, Hk, D, page, out=BF16, causal=1, window=0, scale=None, seed=0, context=None,
                 table=None, pages=None, extra=0, low=None, sharp=1.0):
        rng = np.random.default_rng([41, fmt, len(new), sum(new), max(lengths), Hq, Hk, D, page, seed])
        self.lengths, self.offsets = np.asarray(lengths, np.int64), np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        pages = pages or max(1, sum(-(-max(int(n), 0) // page) for n in lengths)) + 2
        self.table = table_of(rng, lengths, page, pages) if table is None else np.asarray(table, np.int32)
        self.ref = make_cache(rng, fmt, Hk, D, page, lengths, self.table, pages, low)
        self.T, self.out, self.D, self.Hq = int(self.offsets[-1]) + extra, out, D, Hq
        self.ldq, self.ldy = Hq * D + 24, Hq * D + 16
        bits = wl._to_bf16_bits((rng.normal(size=(max(1, self.T), self.ldq)) * sharp).astype(np.float32))
        self.q_np = wl.bf16_bits_to_f32(bits)[:, :Hq * D].reshape(-1, Hq, D)
        self.q = to_dev_bf16(bits)
        self.y = guarded((max(1, self.T), self.ldy), torch.float32 if out == F32 else torch.int16, 9)
        self.scale, self.causal, self.window = D ** -0.5 if scale is None else scale, causal, window
        self.attention = q.make_attention(Hq, self.scale, causal, window)
        self.arrays = [to_dev(a) for a in (*self.ref.codes, *self.ref.scales)]
        self.cache = q.make_cache(fmt, Hk, D, page, pages, *self.arrays)
        self.longest = max(1, int(min(max(lengths), self.table.shape[1] * page)))
        self.sequences = q.make_sequences(len(new), self.T, to_dev(self.offsets), to_dev(self.lengths.astype(np.int32)),
                                          to_dev(self.table), self.table.shape[1], context or self.longest)
        self.work = guarded((q.qlin_cache_attention_workspace_bytes(self.attention, self.cache, self.sequences),),
                            torch.uint8, 0xFF)
        print(f"[attention] fmt={fmt} new={[int(v) for v in new[:8]]} lengths={[int(v) for v in lengths[:8]]} heads={Hq}/{Hk} D={D} page={page} "
              f"out={out} causal={causal} window={window} context={context}", flush=True)

    def run(self, stream=None):
        q.qlin_cache_attention(self.attention, self.cache, self.sequences, self.q, self.ldq, self.y, self.ldy, self.out,
                               self.work, stream=stream)

    def check(self):
        torch.cuda.synchronize()
        check_guards(self.y, self.work, what="qlin_cache_attention")
        full = self.y.cpu().numpy()
        n = self.Hq * self.D
        assert (full[:, n:] == 9).all(), "columns behind the heads changed"
        used = int(self.offsets[-1])
        assert (full[used:] == 9).all(), "rows behind the last sequence changed"
        if used == 0:
            return 0.0
        got = full[:used, :n] if self.out == F32 else wl.bf16_bits_to_f32(full.view(np.uint16)[:used, :n])
        got = got.reshape(used, self.Hq, self.D).astype(np.float64)
        y, W, E, F = oa.attention(self.ref, self.offsets, self.lengths, self.table, self.q_np[:used], self.scale,
                               bool(self.causal), self.window)
        n = np.diff(self.offsets)
        tol = tolerance(y, W, E, F, self.D, self.longest, self.out, np.repeat(n * (self.Hq // self.cache.kv_heads) > 64, n))
        assert np.isfinite(got).all(), f"{np.argwhere(~np.isfinite(got))[:3]} not finite"
        err = np.abs(got - y)
        at = np.unravel_index(np.argmax(err / tol), err.shape)
        assert (err <= tol).all(), f"off by {(err / tol)[at]:.3g} tolerances at {at}: {got[at]} for {y[at]}"
        return float((err / tol).max())


def check(*args, **kw):
    c = Call(*args, **kw)
    c.run()
    worst = c.check()
    print(f"  worst {worst:.3f} of the tolerance", flush=True)


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("fmt,out", [(FP8, BF16), (INT8, F32)])
def test_single_tokens(fmt, out, D, page):
    check(fmt, [1] * 6, [1, 61, 128, 333, 16, 200], 8, 2, D, page, out)


@pytest.mark.parametrize("fmt", [FP8, INT8])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 192, 256])
def test_several_tokens(fmt, out, D):
    check(fmt, [5, 0, 1, 40, 3], [9, 50, 1, 77, 300], 6, 2, D, 32, out)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (4, 4), (5, 1), (16, 1), (17, 1), (40, 2), (64, 8), (24, 3)])
def test_head_groups(Hq, Hk):
    check(FP8, [1, 1, 1], [100, 37, 1], Hq, Hk, 64, 16)
    check(INT8, [7, 2, 0, 1], [100, 37, 20, 5], Hq, Hk, 64, 16, F32)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 255, 256, 257, 511, 513, 1023, 1500])
def test_lengths(n):
    check(INT8, [1], [n], 4, 1, 64, 16, F32)
    check(FP8, [min(n, 33)], [n], 4, 1, 64, 64, F32)


@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 1000, (1 << 31) - 1])
@pytest.mark.parametrize("causal", [0, 1])
def test_windows(window, causal):
    check(FP8, [1, 9, 50, 3], [200, 200, 50, 3], 4, 2, 64, 16, F32, causal, window)


def test_pages_left_behind_a_window_may_be_taken_out():
    window, lengths, new = 40, [300, 130, 41], [1, 20, 1]
    low = [max(0, n - m - window + 1) for n, m in zip(lengths, new)]
    rng = np.random.default_rng(4)
    table = table_of(rng, lengths, 16, 40)
    for s, l in enumerate(low):
        table[s, :l // 16] = -1 if s else 12345678
    for out in (BF16, F32):
        check(FP8, new, lengths, 4, 2, 64, 16, out, window=window, table=table, pages=40, low=low)


@pytest.mark.parametrize("causal", [0, 1])
def test_tokens_that_see_nothing(causal):
    # no page at all; positions before 0; a length of 0 with a token; a negative length
    table = np.array([[-1, -1, -1], [0, 1, 2], [3, 4, 5], [6, 7, 8], [9, 10, 11]])
    check(FP8, [2, 5, 1, 2, 40], [40, 2, 0, -7, 30], 4, 2, 64, 16, F32, causal, table=table, pages=12)
    check(INT8, [20, 30, 1, 2, 60], [40, 2, 0, -7, 30], 4, 2, 64, 16, BF16, causal, table=table, pages=12)


def test_absent_pages_and_lengths_past_the_table():
    table = np.array([[0, -1, 2, 99, 4], [5, 6, -(1 << 31), 8, (1 << 31) - 1], [10, 11, 12, 13, 14]])
    for out in (BF16, F32):
        check(FP8, [1, 4, 2], [77, 80, 1000], 4, 2, 64, 16, out, table=table, pages=15)
        check(FP8, [1, 30, 2], [77, 80, 81], 4, 2, 64, 16, out, table=table, pages=15)
    check(INT8, [1, 1, 1], [(1 << 31) - 1, 70, 1 << 30], 4, 2, 64, 16, table=table, pages=15, context=80)


@pytest.mark.parametrize("context", [1, 100, 4000, 1 << 20, 1 << 30])
def test_the_expected_context_does_not_matter(context):
    check(FP8, [1, 1, 1], [2100, 3, 700], 4, 1, 64, 64, F32, context=context)
    check(FP8, [20, 1, 0], [2100, 3, 700], 4, 1, 64, 64, F32, context=context)


@pytest.mark.parametrize("fmt", [FP8, INT8])
def test_long_contexts(fmt):
    check(fmt, [1], [9000], 8, 2, 128, 128, F32)
    check(fmt, [1, 3], [9000, 5000], 8, 2, 128, 16, BF16, window=7000)


def test_sharp_and_flat_scores():
    check(FP8, [1, 3], [300, 500], 4, 2, 64, 32, F32, sharp=40.0)        # one probability is nearly all
    check(FP8, [1, 3], [300, 500], 4, 2, 64, 32, F32, scale=0.0)
    check(FP8, [1, 3], [300, 500], 4, 2, 64, 32, F32, scale=-0.2)
    check(INT8, [1, 3], [300, 500], 4, 2, 64, 32, F32, sharp=1e-30)


@pytest.mark.parametrize("out", [BF16, F32])
def test_prompts(out):
    check(FP8, [300, 0, 129, 64], [300, 10, 500, 65], 8, 2, 128, 64, out)
    check(INT8, [200], [1000], 16, 4, 64, 16, out, window=150)
    check(FP8, [257], [400], 3, 1, 128, 128, out, causal=0)
    check(INT8, [150], [260], 4, 2, 192, 32, out)
    check(FP8, [150], [260], 4, 2, 256, 32, out)


def test_rows_past_the_last_sequence_and_empty_calls():
    check(FP8, [1, 1, 0], [40, 9, 7], 4, 2, 64, 16, extra=9)
    check(FP8, [0, 0], [40, 9], 4, 2, 64, 16, extra=3)
    check(FP8, [0, 0], [40, 9], 4, 2, 64, 16)


def test_many_sequences():
    rng = np.random.default_rng(6)
    lengths = rng.integers(1, 60, 200)
    new = np.minimum(rng.integers(0, 3, 200), lengths)
    check(FP8, new, lengths, 2, 1, 64, 16)
    check(INT8, [1] * 200, lengths, 2, 1, 64, 16, F32)


def test_padded_batches():
    """Hundreds of sequences without tokens between and behind the others."""
    rng = np.random.default_rng(9)
    for B, live in ((300, [0, 7, 299]), (300, [150]), (700, [3, 64, 65, 690]), (5000, [17, 2400, 4999])):
        new, lengths = np.zeros(B, int), np.zeros(B, int)
        lengths[rng.integers(0, B, 20)] = 30
        for s in live:
            new[s], lengths[s] = 1 + s % 3, 600 + s % 7
        check(FP8, new, lengths, 8, 4, 64, 16, F32, extra=4)
        new[live[0]] = 200
        check(FP8, new, lengths, 8, 4, 64, 16, BF16)


def test_offsets_are_clamped():
    c = Call(INT8, [4, 6, 0, 0], [40, 60, 1, 1], 4, 2, 64, 16)
    c.run()
    torch.cuda.synchronize()
    want = c.y.clone()
    c.y.fill_(9)
    c.sequences.tensors[0].copy_(torch.tensor([-3, 4, 1 << 30, 8, -(1 << 31)], dtype=torch.int32))
    c.run()
    torch.cuda.synchronize()
    check_guards(c.y, c.work)
    assert torch.equal(c.y, want)


def test_offsets_that_go_back():
    """Sequences that overlap in their rows: whose result stays is open, but nothing else is written."""
    for B, T in ((100, 50), (300, 200), (40, 7)):
        new = np.zeros(B, int)
        new[0] = T
        c = Call(FP8, new, np.full(B, 230), 16, 4, 64, 16, extra=5)
        offsets = torch.tensor([0, T] * (B // 2) + [0], dtype=torch.int32)
        c.sequences.tensors[0].copy_(offsets)
        c.run()
        torch.cuda.synchronize()
        check_guards(c.y, c.work, what="qlin_cache_attention")
        full = c.y.cpu().numpy()
        assert (full[T:] == 9).all() and (full[:, c.Hq * c.D:] == 9).all()
        got = wl.bf16_bits_to_f32(full.view(np.uint16)[:T, :c.Hq * c.D])
        assert np.isfinite(got).all()


def test_the_same_bits_every_time_and_with_other_sequences_beside():
    c = Call(FP8, [1, 1], [3000, 1200], 8, 2, 128, 64, F32)
    c.run()
    torch.cuda.synchronize()
    want = c.y.clone()
    for _ in range(5):
        c.work.fill_(0xFF)
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(c.y, want)


def test_graphs_follow_their_arrays():
    """Captured and replayed with other lengths, tables and queries; two graphs
    share one workspace, with eager calls between."""
    calls = [Call(FP8, [1, 1, 1], [3000, 70, 500], 8, 2, 64, 16, F32), Call(INT8, [4, 2], [900, 2000], 8, 2, 64, 16, BF16)]
    work = torch.full((max(c.work.nbytes for c in calls),), 0xFF, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = []
    for c in calls:
        c.work = work
        q.qlin_graph_begin(stream)
        c.run(stream)
        graphs.append(q.qlin_graph_end(stream))
    for step in range(3):
        for c, g in zip(calls, graphs):
            c.y.fill_(9)
            torch.cuda.synchronize()
            q.qlin_graph_launch(g, stream)
            torch.cuda.synchronize()
            c.check()
            eager = c.y.clone()
            c.y.fill_(9)
            c.run()
            torch.cuda.synchronize()
            assert torch.equal(c.y, eager)
        for c in calls:                              # the next step: shorter sequences
            c.lengths = c.lengths - 13 * (step + 1)
            c.sequences.tensors[1].copy_(torch.from_numpy(c.lengths.astype(np.int32)))
    for g in graphs:
        q.qlin_graph_destroy(g)


def test_pools_past_32_bits():
    """Sequences in the last pages of a pool of more than 4 GiB of codes."""
    H, D, page = 8, 256, 128
    pages = (1 << 32) // (H * D * page) + 40
    small = Call(FP8, [1, 2], [200, 400], 8, 8, D, page, F32)
    codes = [torch.full((pages, H, page * D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((pages, H), float("nan"), device="cuda") for _ in range(2)]
    moved = pages - small.ref.pages
    for kv in range(2):
        codes[kv][moved:].copy_(small.arrays[kv])
        scales[kv][moved:].copy_(small.arrays[2 + kv])
    small.cache = q.make_cache(FP8, H, D, page, pages, *codes, *scales)
    table = small.sequences.tensors[2]
    table[table >= 0] += moved
    small.run()
    small.check()


def scaled(c, kv, factor):
    """The pages' scales times factor(page number in its sequence, sequence)."""
    for s in range(len(c.lengths)):
        for which in range(c.table.shape[1]):
            p = c.ref.page_of(c.table, s, which * c.ref.page)
            if p >= 0:
                c.ref.scales[kv][p] *= np.float32(factor(which, s))
    c.arrays[2 + kv].copy_(torch.from_numpy(c.ref.scales[kv]))


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("name,factor", [
    ("growing", lambda w, s: 2.0 ** (3 * w)), ("falling", lambda w, s: 2.0 ** (-3 * w)),
    ("far apart", lambda w, s: 2.0 ** (20 if w % 3 == 1 else 0)), ("zeros", lambda w, s: 0.0 if w % 2 else 1.0),
    ("all zeros", lambda w, s: 0.0), ("tiny", lambda w, s: 2.0 ** -60), ("huge", lambda w, s: 2.0 ** 60)])
def test_value_scales_of_any_size(name, factor, out):
    for new, page in (([300, 20], 16), ([1, 3], 16), ([280, 70], 64)):
        c = Call(FP8 if page == 16 else INT8, new, [400, 130], 8, 2, 64 if page == 16 else 128, page, out)
        scaled(c, 1, factor)
        c.run()
        c.check()


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("name,factor", [
    ("small between", lambda w, s: 2.0 ** (-110 if w % 3 == 1 else 0)), ("small first", lambda w, s: 2.0 ** (-110 if w == 0 else 0)),
    ("large last", lambda w, s: 2.0 ** (100 if w == 3 else 0)), ("both ends", lambda w, s: 2.0 ** (-90 if w % 2 else 60)),
    ("steps of 2^40", lambda w, s: 2.0 ** (90 - 40 * (w % 5)))])
def test_value_scales_over_the_whole_range(name, factor, out):
    for new, page in (([300, 20], 16), ([280, 70], 64)):
        c = Call(FP8 if page == 16 else INT8, new, [400, 330], 8, 2, 64 if page == 16 else 128, page, out)
        scaled(c, 1, factor)
        c.run()
        c.check()


@pytest.mark.parametrize("out", [BF16, F32])
def test_key_scales_of_zero(out):
    for new in ([300, 20], [1, 3]):
        c = Call(FP8, new, [400, 130], 8, 2, 64, 16, out, window=200)
        scaled(c, 0, lambda w, s: 0.0 if w % 2 else 1.0)
        c.run()
        c.check()


@pytest.mark.parametrize("causal,window", [(1, 0), (0, 0), (1, 70), (0, 70), (1, 1)])
def test_long_and_short_sequences_together(causal, window):
    new, lengths = [1, 200, 0, 7, 1, 129, 33], [700, 200, 9, 1000, 3, 400, 33]
    check(FP8, new, lengths, 8, 2, 64, 16, BF16, causal, window, extra=5)
    check(INT8, new, lengths, 20, 2, 128, 32, F32, causal, window)
    check(FP8, new, lengths, 6, 2, 192, 64, BF16, causal, window)
    check(INT8, new, lengths, 6, 2, 256, 128, BF16, causal, window)


@pytest.mark.parametrize("D", [64, 128, 192, 256])
def test_long_contexts_of_many_rows(D):
    """Units of many rows whose tokens several workgroups share."""
    check(FP8, [130], [2500], 5, 1, D, 64, BF16)
    check(INT8, [70, 1, 66], [2300, 40, 1100], 8, 1, D, 16, F32, window=1500)
    check(FP8, [70, 66], [1 + 2300, 1100], 16, 1, D, 128, BF16, causal=0)


@pytest.mark.parametrize("out", [BF16, F32])
def test_one_sequence_of_some_rows_over_many_tokens(out):
    for fmt, new, page in ((FP8, 9, 64), (INT8, 16, 16), (FP8, 8, 128)):
        check(fmt, [new], [5100], 32, 8, 64, page, out)
        check(fmt, [new], [5100], 32, 8, 128, page, out, window=2000)


def test_many_rows_that_see_nothing():
    table = np.array([[-1] * 12, [0, 1, 2] + [-1] * 9, list(range(3, 15))])
    check(FP8, [100, 200, 90], [150, 20, 180], 8, 1, 64, 16, F32, table=table, pages=16)
    check(FP8, [100, 200, 90], [150, 20, 180], 8, 1, 64, 16, BF16, table=table, pages=16)
