// qlin_sequences.h -- device-side view of a call's sequences: the rows of each,
// the positions they have, and which sequence a workgroup's unit belongs to.
#pragma once

#include "qlin_device.h"

namespace qlin {

constexpr int kMaxPosition = 1 << 30;   // positions stay far from the end of 32 bits

struct Sequence {
    int first, n;     // rows [first, first + n) of the call's tensors
    int start;        // position of the first (may be negative)
    int length;       // positions that the page table can hold, of the sequence's
};

__device__ __forceinline__ Sequence sequence_at(const CacheArgs &c, int s) {
    Sequence q;
    const int lo = min(max(c.offsets[s], 0), c.T), hi = min(max(c.offsets[s + 1], 0), c.T);
    const int length = max(c.lengths[s], 0);
    q.first = lo;
    q.n = max(hi - lo, 0);
    q.start = length - q.n;
    q.length = (int)min((int64_t)min(length, kMaxPosition), (int64_t)c.max_pages << c.page_shift);
    return q;
}

// sum of v over the lanes up to and with this one
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);    // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);    // row_shr:2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);    // row_shr:4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);    // row_shr:8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast:15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // row_bcast:31 into rows 2 and 3
    return v;
}

// The sequence that unit u belongs to, where sequence s has count(s) units, and
// u's number among its units (in *within); -1: u is past the last.  One pass of a
// wave over 64 sequences at a time: a load, a scan of six steps and a ballot.
template <typename F>
__device__ __forceinline__ int unit_sequence(const CacheArgs &c, int u, F count, int *within) {
    const int lane = threadIdx.x & 63;
    int64_t base = 0;                              // units before sequence s0
    for (int s0 = 0; s0 < c.B; s0 += 64) {
        const int s = s0 + lane;
        const int n = s < c.B ? min(count(sequence_at(c, s)), 1 << 24) : 0;   // 64 of them stay in 32 bits
        const int upto = wave_scan(n);
        const uint64_t past = __ballot(base + upto > u);
        if (past) {
            const int l = __builtin_ctzll(past);
            *within = u - (int)base - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(n, l));
            return s0 + l;
        }
        base += __builtin_amdgcn_readlane(upto, 63);
    }
    return -1;
}

// pages that a sequence's own tokens of the call touch, and the first of them
__device__ __forceinline__ int touched_pages(const CacheArgs &c, const Sequence &q, int *first) {
    const int lo = max(q.start, 0);
    *first = lo >> c.page_shift;
    return q.n > 0 && q.length > lo ? ((q.length - 1) >> c.page_shift) - *first + 1 : 0;
}

// the pool's page that holds a sequence's c-th, or -1
__device__ __forceinline__ int pool_page(const CacheArgs &c, int s, int page) {
    const int p = page < c.max_pages ? c.table[(int64_t)s * c.max_pages + page] : -1;
    return (unsigned)p < (unsigned)c.pages ? p : -1;
}

}  // namespace qlin
