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

// v and the one that a lane permutation brings (0 where it brings none)
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ int64_t add_dpp(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROW_MASK, 0xF, ROW_MASK == 0xF);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(v >> 32), CTRL, ROW_MASK, 0xF, ROW_MASK == 0xF);
    return v + (int64_t)((uint64_t)hi << 32 | lo);
}

// sum of v over the lanes up to and with this one
__device__ __forceinline__ int64_t wave_scan(int64_t v) {
    v = add_dpp<0x111, 0xF>(v);    // row_shr:1
    v = add_dpp<0x112, 0xF>(v);    // row_shr:2
    v = add_dpp<0x114, 0xF>(v);    // row_shr:4
    v = add_dpp<0x118, 0xF>(v);    // row_shr:8
    v = add_dpp<0x142, 0xA>(v);    // row_bcast:15 into rows 1 and 3
    return add_dpp<0x143, 0xC>(v); // row_bcast:31 into rows 2 and 3
}
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
    return v;
}

// the sequence that a lane has, in scalar registers
__device__ __forceinline__ Sequence lane_of(const Sequence &q, int lane) {
    return Sequence{__builtin_amdgcn_readlane(q.first, lane), __builtin_amdgcn_readlane(q.n, lane),
                    __builtin_amdgcn_readlane(q.start, lane), __builtin_amdgcn_readlane(q.length, lane)};
}

// A wave takes 64 PER sequences at a time, PER a lane: their loads together, a scan
// of six steps and a ballot.  A call has fewer than 2^24 units, so larger sums are of
// offsets that go back; as clamped they stay in 32 bits, and a unit among its
// sequence's.
template <int PER, typename F>
__device__ __forceinline__ int unit_sequence_by(const CacheArgs &c, int64_t u, F count, int *within) {
    const int lane = threadIdx.x & 63;
    int64_t base = 0;                              // units before sequence s0
    for (int s0 = 0; s0 < c.B; s0 += 64 * PER) {
        int n[PER], all = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int s = s0 + PER * lane + i;
            n[i] = s < c.B ? min((int)count(sequence_at(c, s)), 1 << 24) : 0;
            all += n[i];
        }
        all = min(all, 1 << 24);
        const int upto = wave_scan(all);
        const uint64_t past = __ballot(base + upto > u);
        if (past) {
            const int l = __builtin_ctzll(past);
            int rest = (int)(u - base) - __builtin_amdgcn_readlane(upto, l) + __builtin_amdgcn_readlane(all, l);
            int s = s0 + PER * l;
#pragma unroll
            for (int i = 0; i + 1 < PER; ++i) {
                const int here = __builtin_amdgcn_readlane(n[i], l);
                if (rest < here) break;
                rest -= here;
                ++s;
            }
            *within = rest;
            return s;
        }
        base += __builtin_amdgcn_readlane(upto, 63);
    }
    return -1;
}

// The sequence that unit u belongs to, where sequence s has count(s) units, and
// u's number among its units (in *within); -1: u is past the last.
template <typename F>
__device__ __forceinline__ int unit_sequence(const CacheArgs &c, int64_t u, F count, int *within) {
    return c.B <= 64 ? unit_sequence_by<1>(c, u, count, within) : unit_sequence_by<4>(c, u, count, within);
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
