"""The 8-bit cache on the GPU against the oracle, every byte and scale of the
pool equal after each call (the steps are defined in 32 bits)."""
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


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.lib()


class Both:
    """A cache on the device and the oracle's, filled with NaN codes and scales."""

    def __init__(self, fmt, H, D, page, pages, seed=0):
        self.fmt, self.H, self.D, self.page, self.pages = fmt, H, D, page, pages
        self.ref = oa.Cache(fmt, H, D, page, pages)
        self.codes = [guarded((pages, H, page * D), torch.uint8, 0x7F) for _ in range(2)]
        self.scales = [guarded((pages, H), torch.float32, float("nan")) for _ in range(2)]
        self.cache = q.make_cache(fmt, H, D, page, pages, *self.codes, *self.scales)
        self.rng = np.random.default_rng([31, fmt, H, D, page, pages, seed])

    def rows(self, T, type_, amplitude=1.0):
        """(device rows in a wider tensor, their fp32 values) of keys and values."""
        ld = 3 * self.H * self.D + 8
        x = (self.rng.normal(size=(T, ld)) * amplitude).astype(np.float32)
        if type_ == BF16:
            bits = wl._to_bf16_bits(x)
            x, dev = wl.bf16_bits_to_f32(bits), to_dev_bf16(bits)
        else:
            dev = to_dev(x)
        n = self.H * self.D
        cut = [slice(n, 2 * n), slice(2 * n, 3 * n)]
        return [dev[:, c] for c in cut], [x[:, c].reshape(T, self.H, self.D) for c in cut], ld

    def sequences(self, new, lengths, table, T=None, offsets=None):
        offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int32) if offsets is None else offsets
        T = int(offsets[-1]) if T is None else T
        lengths, table = np.asarray(lengths, np.int32), np.asarray(table, np.int32)
        return offsets, lengths, table, q.make_sequences(len(lengths), T, to_dev(offsets), to_dev(lengths), to_dev(table),
                                                         table.shape[1], min(max(1, int(lengths.max(initial=1))), 1 << 30))

    def append(self, new, lengths, table, type_=BF16, amplitude=1.0, extra=0, stream=None):
        offsets, lengths, table, s = self.sequences(new, lengths, table, sum(new) + extra)
        dev, x, ld = self.rows(max(1, s.tokens), type_, amplitude)
        print(f"[append] fmt={self.fmt} H={self.H} D={self.D} page={self.page} new={list(new)[:9]} "
              f"lengths={lengths.tolist()[:9]} type={type_}", flush=True)
        q.qlin_cache_append(self.cache, s, dev[0], ld, dev[1], ld, type_, stream=stream)
        torch.cuda.synchronize()
        self.ref.append(offsets, lengths, table, *x)
        self.check("append")

    def check(self, what):
        check_guards(*self.codes, *self.scales, what=what)
        for kv in range(2):
            got = self.scales[kv].cpu().numpy()
            assert np.array_equal(got.view(np.uint32)[~np.isnan(got)], self.ref.scales[kv].view(np.uint32)[~np.isnan(got)])
            assert np.array_equal(np.isnan(got), np.isnan(self.ref.scales[kv])), f"{what}: scales of {'kv'[kv]}"
            codes = self.codes[kv].cpu().numpy()
            bad = np.argwhere(codes != self.ref.codes[kv])
            assert len(bad) == 0, f"{what}: {len(bad)} codes of {'kv'[kv]} differ, first at {bad[0]}"

    def read(self, new, lengths, table, type_=BF16, extra=0, which="kv"):
        offsets, lengths, table, s = self.sequences(new, lengths, table, sum(new) + extra)
        n, T = self.H * self.D, max(1, s.tokens)
        kind = torch.float32 if type_ == F32 else torch.int16
        out = [guarded((T, n + 8), kind, 9), guarded((T, n + 16), kind, 9)]
        q.qlin_cache_read(self.cache, s, out[0] if "k" in which else None, n + 8, out[1] if "v" in which else None, n + 16,
                          type_)
        torch.cuda.synchronize()
        check_guards(*out, what="read")
        for kv in range(2):
            want = np.full((T, n), 9, dtype=np.float32 if type_ == F32 else np.int16)
            if "kv"[kv] in which:
                for i in range(len(lengths)):
                    start = int(lengths[i]) - int(offsets[i + 1] - offsets[i])
                    for t in range(offsets[i], offsets[i + 1]):
                        x = self.ref.token(kv, table, i, start + t - int(offsets[i]))
                        if x is not None:
                            want[t] = x.ravel() if type_ == F32 else wl._to_bf16_bits(x.ravel()).view(np.int16)
            got = out[kv].cpu().numpy()
            assert np.array_equal(got[:, :n].view(np.uint8), want.view(np.uint8)), f"read of {'kv'[kv]}"
            assert (got[:, n:] == 9).all()


def table_of(rng, lengths, page, pages, width=None):
    """Distinct pages in random order, -1 behind them."""
    held = [-(-int(n) // page) for n in lengths]
    table = np.full((len(lengths), width or max(held) + 1), -1, dtype=np.int32)
    free = rng.permutation(pages)[:sum(held)]
    assert len(free) == sum(held)
    for i, n in enumerate(held):
        table[i, :n], free = free[:n], free[n:]
    return table


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("fmt,type_", [(FP8, BF16), (INT8, F32)])
def test_prompts_then_tokens(fmt, type_, D, page):
    b = Both(fmt, 2, D, page, 24)
    lengths = np.array([page + 7, 5, 2 * page, 1])
    table = table_of(b.rng, lengths + 2 * page, page, 24)
    b.append(lengths, lengths, table, type_)
    for step, amplitude in enumerate((0.5, 3.0, 1.0, 9.0)):          # scales that stay, and that grow
        lengths = lengths + 1
        b.append([1] * 4, lengths, table, type_, amplitude)
    lengths = lengths + [3, 0, page + 5, 2]
    b.append([3, 0, page + 5, 2], lengths, table, type_, 11.0)
    b.read(lengths, lengths, table, type_)
    b.read([2, 0, page, 1], lengths, table, type_)


@pytest.mark.parametrize("fmt", [FP8, INT8])
@pytest.mark.parametrize("type_", [BF16, F32])
def test_formats_and_types(fmt, type_):
    b = Both(fmt, 8, 128, 64, 40)
    lengths = np.array([100, 64, 1, 333, 63])
    table = table_of(b.rng, lengths + 4, 64, 40)
    b.append(lengths, lengths, table, type_)
    b.append([2, 0, 1, 4, 1], lengths + [2, 0, 1, 4, 1], table, type_, 4.0)
    b.read(lengths, lengths, table, F32)
    b.read(lengths, lengths, table, BF16)
    b.read([3, 3, 1, 3, 3], lengths, table, BF16, which="k", extra=5)
    b.read([3, 3, 1, 3, 3], lengths, table, F32, which="v")


def test_drafts_are_stored_over():
    b = Both(FP8, 2, 64, 16, 8)
    table = table_of(b.rng, [40], 16, 8)
    b.append([14], [14], table)
    b.append([5], [19], table, amplitude=6.0)       # two of the five stay
    b.append([5], [21], table, amplitude=1.0)
    b.append([1], [17], table, amplitude=0.1)       # page 1 starts anew
    b.read([17], [17], table)


@pytest.mark.parametrize("fmt", [FP8, INT8])
def test_extremes(fmt):
    b = Both(fmt, 1, 64, 16, 6)
    table = table_of(b.rng, [60], 16, 6)
    b.append([4], [4], table, F32, 0.0)             # a page of zeros: scale 0
    b.append([1], [5], table, F32, 1e-30)
    b.append([1], [6], table, F32, 1e-25)
    b.append([1], [7], table, F32, 1.0)
    b.append([1], [8], table, F32, 1e30)
    b.append([3], [11], table, F32, 1e-44)
    b.append([29], [40], table, F32, 1e-38)
    b.read([40], [40], table, F32)


def test_many_sequences():
    b = Both(INT8, 1, 64, 16, 900)
    lengths = b.rng.integers(1, 40, 300)
    new = np.minimum(b.rng.integers(0, 9, 300), lengths)
    table = table_of(b.rng, lengths, 16, 900)
    old = lengths - new
    b.append(old, old, table, F32)
    b.append(new, lengths, table, F32, 2.0)
    b.read(new, lengths, table, F32, extra=3)


@pytest.mark.parametrize("fmt", [FP8, INT8])
@pytest.mark.parametrize("type_", [BF16, F32])
@pytest.mark.parametrize("D,page", [(64, 32), (128, 128), (192, 16), (256, 64)])
def test_few_tokens_beside_many(fmt, type_, D, page):
    """Calls on both sides of the average at which a wave has a page, not a workgroup."""
    b = Both(fmt, 3, D, page, 100)
    lengths = np.array([50, 3, 90, 20, 1, 0])
    table = table_of(b.rng, lengths + 60, page, 100)
    b.append(lengths, lengths, table, type_)
    for new, amplitude in (([40, 0, 1, 3, 2, 1], 5.0), ([1, 1, 0, 1, 1, 1], 2.0), ([0, 2, 3, 1, 0, 1], 20.0),
                           ([9, 9, 9, 9, 9, 9], 50.0)):
        lengths = lengths + new
        b.append(new, lengths, table, type_, amplitude)
    b.append([2, 30, 2, 2, 2, 2], lengths, table, type_, 60.0)       # stored over
    b.read(lengths, lengths, table, type_)


def test_absent_tokens_and_bad_tables():
    b = Both(FP8, 2, 64, 16, 8)
    table = np.array([[3, -1, 5], [8, 1 << 30, -(1 << 31)], [1, 2, 4], [0, 7, 6]], dtype=np.int32)
    b.append([0, 0, 0, 44], [40, 20, 9, 44], table)      # what the last one holds already
    # pages missing in the middle; none at all; positions before 0; more tokens than the table holds
    b.append([40, 20, 12, 8], [40, 20, 9, 52], table)
    b.read([40, 20, 12, 8], [40, 20, 9, 52], table, extra=2)
    b.append([1, 1, 1, 1], [-5, 0, -(1 << 31), (1 << 31) - 1], table)
    b.read([1, 1, 1, 1], [-5, 0, -(1 << 31), (1 << 31) - 1], table)


def test_offsets_are_clamped():
    """Whatever the offsets hold, nothing outside the tensors is touched."""
    b = Both(INT8, 1, 64, 16, 8)
    table = np.arange(8, dtype=np.int32).reshape(4, 2)
    dev, x, ld = b.rows(10, BF16)
    offsets = np.array([-3, 4, 1 << 30, 8, -(1 << 31)], dtype=np.int32)      # as clamped: 0, 4, 10, 8, 0
    s = q.make_sequences(4, 10, to_dev(offsets), to_dev(np.array([4, 6, 1, 1], np.int32)), to_dev(table), 2, 10)
    q.qlin_cache_append(b.cache, s, dev[0], ld, dev[1], ld)
    torch.cuda.synchronize()
    b.ref.append([0, 4, 10, 10, 10], [4, 6, 1, 1], table, *x)
    b.check("append")


def test_offsets_that_go_back():
    """Two sequences that take the same rows, into pages of their own."""
    b = Both(FP8, 2, 64, 16, 12)
    table = np.arange(12, dtype=np.int32).reshape(3, 4)
    dev, x, ld = b.rows(40, BF16)
    s = q.make_sequences(3, 40, to_dev(np.array([0, 40, 0, 40], np.int32)), to_dev(np.array([40, 9, 40], np.int32)),
                         to_dev(table), 4, 40)
    q.qlin_cache_append(b.cache, s, dev[0], ld, dev[1], ld)
    torch.cuda.synchronize()
    for i in (0, 2):
        b.ref.append([0, 40], [40], table[i:i + 1], *x)
    # a call of 40 tokens has 40 / 16 + 2 x 3 page places at most: the second's six fit too
    b.check("append")


def test_rows_past_the_last_sequence_and_empty_calls():
    b = Both(FP8, 2, 64, 16, 8)
    table = table_of(b.rng, [20, 20], 16, 8)
    b.append([17, 0], [17, 0], table)
    b.append([3, 2], [20, 2], table, extra=7)
    b.read([3, 2], [20, 2], table, extra=7)
    b.append([0, 0], [20, 2], table, extra=4)
    b.append([0, 0], [20, 2], table)


def test_on_another_stream_and_long_pools():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = Both(INT8, 2, 64, 32, 30)
    table = table_of(b.rng, [200, 33], 32, 30)
    torch.cuda.synchronize()
    b.append([200, 33], [200, 33], table, stream=s)


def test_codes_past_32_bits():
    """The last pages of a pool of more than 4 GiB of codes."""
    H, D, page = 8, 256, 128
    pages = (1 << 32) // (H * D * page) + 40
    codes = [torch.zeros(pages * H * page * D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(pages, H, device="cuda") for _ in range(2)]
    cache = q.make_cache(INT8, H, D, page, pages, *codes, *scales)
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
    n = 300
    rng = np.random.default_rng(8)
    x = torch.from_numpy(rng.integers(-127, 128, (n, H * D)).astype(np.float32)).cuda()
    x[::50, ::D] = 127.0                            # every 50th row: each page has one, so its scale is 1
    i32 = dict(dtype=torch.int32, device="cuda")
    s = q.make_sequences(1, n, torch.tensor([0, n], **i32), torch.tensor([n], **i32), table, 3, n)
    q.qlin_cache_append(cache, s, x, H * D, -x, H * D, F32)
    k, v = torch.zeros_like(x), torch.zeros_like(x)
    q.qlin_cache_read(cache, s, k, H * D, v, H * D, F32)
    assert torch.equal(k, x) and torch.equal(v, -x)
    assert torch.equal(scales[0][table[0].long()], torch.ones(3, H, device="cuda"))
    per = H * page * D
    assert all(int(c[per:-2 * per].count_nonzero()) == 0 for c in codes)
