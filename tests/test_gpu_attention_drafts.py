"""Drafts: a few tokens of every sequence, around the sizes at which a call takes other units or
another kernel."""
import time

import numpy as np
import pytest
import torch

import skinny_bit_gemm_amd as q
from test_gpu_attention import BF16, F32, FP8, INT8, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.lib()


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("out", [BF16, F32])
def test_drafts_around_the_rules(D, out):
    rng = np.random.default_rng(12)
    for new in ([4] * 21, [4] * 22, [5] * 16, [3] * 30 + [90], [1] * 40 + [80], [0, 4] * 20, [8] * 11 + [9],
                [16] * 6 + [17], [15, 16, 17, 1, 0, 33]):
        lengths = [n + int(rng.integers(0, 200)) for n in new]
        check(FP8 if len(new) % 2 else INT8, new, lengths, 8, 1, D, 16, out)


def test_four_times_the_sequences_take_less_than_four_times_the_time():
    """The codes of a sequence are read once for all rows of its draft, however many sequences there
    are (16 sequences 38 us, 64 of them 98; 175 where they were read twice)."""
    H, G, D, page, n, new = 8, 8, 128, 64, 4096, 4
    dev = {"device": "cuda"}
    codes = [torch.zeros(64 * n * H * D, dtype=torch.uint8, **dev) for _ in range(2)]
    scales = [torch.ones(64 * n // page, H, **dev) for _ in range(2)]
    cache = q.make_cache(FP8, H, D, page, 64 * n // page, *codes, *scales)
    table = torch.randperm(64 * n // page, generator=torch.Generator().manual_seed(0)).to(torch.int32).view(64, -1).cuda()
    a = q.make_attention(H * G, D ** -0.5)
    calls = {}
    for B in (16, 64):
        offsets = torch.arange(0, new * B + 1, new, dtype=torch.int32, **dev)
        seqs = q.make_sequences(B, new * B, offsets, torch.full((B,), n, dtype=torch.int32, **dev), table[:B], n // page, n)
        x = torch.zeros(new * B, H * G * D, dtype=torch.bfloat16, **dev)
        work = torch.empty(max(16, q.qlin_cache_attention_workspace_bytes(a, cache, seqs)), dtype=torch.uint8, **dev)
        calls[B] = (seqs, x, torch.empty_like(x), work)

    def us(B, reps=200):
        seqs, x, y, work = calls[B]
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(reps):
            q.qlin_cache_attention(a, cache, seqs, x, H * G * D, y, H * G * D, BF16, work)
        torch.cuda.synchronize()
        return (time.perf_counter() - t) / reps * 1e6

    took = {B: [] for B in calls}
    for _ in range(7):                                   # in turn; the first warms up
        for B in calls:
            took[B].append(us(B))
    few, many = (min(took[B][1:]) for B in (16, 64))
    print(f"16 sequences {few:.1f} us, 64 {many:.1f}")
    assert many < 3.5 * few
