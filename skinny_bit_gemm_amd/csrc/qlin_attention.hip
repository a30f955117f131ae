// qlin_attention.hip -- attention over the paged 8-bit cache: sequences with few
// query rows, the join of what was cut, and the plan of a call.
//
// Probabilities enter the second product as two bf16 terms (16 bits of mantissa;
// three, 24 bits, where y is fp32): one term alone costs as much again as the
// rounding of y, and the codes' stream, which bounds these calls, hides the rest.
#include <algorithm>

#include "qlin_attention.h"

namespace qlin {

namespace {

constexpr int kMostWorkers = 768;
constexpr int64_t kMostSteps = (int64_t)1 << 51;
constexpr int kStep = 128;         // tokens: two tiles of 16 for each wave

// ------------------------------------------------------------ few rows a sequence
//
// The cached tokens of every unit, for every key head, are one long line of steps
// of kStep tokens, and each workgroup takes an equal share of it: the codes are
// what bounds the call, so all compute units read the same number of them,
// however the lengths differ.  A unit that lies in one share is written at once;
// of one that is cut, each workgroup leaves its sums, and join_kernel adds them.
// Where contexts are expected to be short, a unit is one step of any length: none
// is cut, and the second launch is left out (one sequence of 500 tokens 7.7 us, 9.8
// with it; of 1000 the other way round, 12.2 and 10.5).
//
// 64 sequences of 300 to 16384 tokens, 64 query heads over 8 of 128, e4m3 (534 MB of
// codes): 100 us a call, 93 traced for this kernel, 5.7 TB/s; equal parts of each sequence
// instead, 164.  131071 tokens of one sequence, 269 MB: 51 us.  What the steps
// measured: codes of the next step asked for while this one is multiplied, and their
// stream with the non-temporal policy, each 10 %.
// a / b, both not negative; 64-bit divisions take some 100 instructions
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return (a | b) >> 32 == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

struct SequenceWork {
    int tiles, tile0, steps;       // row tiles; first tile of 16 tokens, and steps of each
    __device__ __forceinline__ int64_t all() const { return (int64_t)tiles * steps; }
};
template <int ROWS>
__device__ __forceinline__ SequenceWork sequence_work(const AttentionLaunch &a, const Sequence &q) {
    SequenceWork w = {0, 0, 0};
    if (q.n == 0 || (int64_t)q.n * a.group > a.few_rows) return w;
    const Seen first = seen_by(a, q, 0), last = seen_by(a, q, q.n - 1);
    w.tiles = (q.n * a.group + ROWS - 1) / ROWS;
    w.tile0 = first.lo / kTile;
    w.steps = last.up > first.lo && !a.whole ? (last.up - w.tile0 * kTile + kStep - 1) / kStep : 1;
    return w;
}

// What the workgroups find their shares with.
struct Shares {
    int64_t sums[256];             // steps (for one head) of the sequences up to and with each thread's
    int64_t waves[4];
    Sequence first[256];           // each thread's first sequence
};

// Threads have B / 256 sequences each, in order.  Sums over 2^51 are of offsets that go back;
// as clamped, products with the heads stay in 64 bits, and a search ends.
template <int ROWS>
__device__ __forceinline__ void sum_steps(const AttentionLaunch &a, Shares &sh) {
    const int tid = threadIdx.x, per = (a.c.B + 255) / 256;
    int64_t v = 0;
    const int from = tid * per, to = min(a.c.B, from + per);
    if (from < to) {
        const Sequence q = sequence_at(a.c, from);
        sh.first[tid] = q;
        v = sequence_work<ROWS>(a, q).all();
    }
#pragma unroll 4
    for (int s = from + 1; s < to; ++s) v = min(v + sequence_work<ROWS>(a, sequence_at(a.c, s)).all(), kMostSteps);
    v = wave_scan(v);
    if ((tid & 63) == 63) sh.waves[tid >> 6] = v;
    __syncthreads();
    for (int w = 0; w < tid >> 6; ++w) v += sh.waves[w];
    sh.sums[tid] = min(v, kMostSteps);
    __syncthreads();
}

// RT: tiles of 16 query rows; all waves have the same rows and take groups of NT
// tiles of tokens in turn, so a code is read and converted once for all rows.
template <int D, int FMT, int TERMS, int RT>
__global__ __launch_bounds__(64 * kWaves, RT == 1 || D <= 128 ? 2 : 1) void attention_kernel(AttentionLaunch a) {
    constexpr int ROWS = 16 * RT, J = D / 64, DT = D / 16, NT = kStep / (kWaves * kTile);
    constexpr int AHEAD = 64 / NT;              // groups whose pages a wave looks up at once
    constexpr bool F32 = TERMS == 3;
    __shared__ float merge[kWaves][16][D + 4];
    __shared__ float2 merge_ml[kWaves][16];
    const CacheArgs &c = a.c;
    const int worker = blockIdx.x;
    const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    // this worker's share: of up to 64 sequences each wave finds it by itself, a sequence a lane
    Shares &sh = *reinterpret_cast<Shares *>(merge);
    static_assert(sizeof(Shares) <= sizeof(merge), "they share the LDS");
    const bool by_wave = c.B <= 64;
    Sequence lane_q = {};
    int64_t lane_all = 0, lane_upto = 0, per_head;
    if (by_wave) {
        if (lane < c.B) lane_q = sequence_at(c, lane);
        lane_all = sequence_work<ROWS>(a, lane_q).all();
        lane_upto = wave_scan(lane_all);
        per_head = readlane(lane_upto, 63);
    } else {
        sum_steps<ROWS>(a, sh);
        per_head = uniform(sh.sums[255]);
    }
    const int64_t steps = per_head * c.heads;
    const int64_t share = quotient(steps + a.workers - 1, a.workers);
    int64_t at = worker * share;
    const int64_t end = min(steps, at + share);
    if (threadIdx.x == 0 && !a.whole) a.cuts[worker].parts = 0;
    if (at >= end) return;
    int head = (int)quotient(at, per_head), seq;
    int64_t begin = (int64_t)head * per_head;   // of the sequence, and then of the unit
    Sequence sq;
    // among 64 sequences from `from` on, a lane each, the one that has step `at`
    auto find_lane = [&](int from, const Sequence &q, int64_t all, int64_t upto) {
        const uint64_t past = __ballot(begin + upto > at);
        if (past == 0) {
            begin += readlane(upto, 63);
            return false;
        }
        const int l = __builtin_ctzll(past);
        begin += readlane(upto - all, l);
        seq = from + l;
        sq = lane_of(q, l);
        return true;
    };
    if (by_wave) {
        find_lane(0, lane_q, lane_all, lane_upto);
    } else {
        int block = 0;                          // the thread whose sequences have it
#pragma unroll
        for (int i = 0; i < 4; ++i) block += __popcll(__ballot(sh.sums[64 * i + lane] <= at - begin));
        begin += block ? uniform(sh.sums[block - 1]) : 0;
        const int per = (c.B + 255) / 256;
        seq = block * per;
        sq = uniform(sh.first[block]);
        for (int from = seq; per > 1; from += 64) {
            const int s = from + lane;
            Sequence q = {};
            if (s < c.B) q = sequence_at(c, s);
            const int64_t all = sequence_work<ROWS>(a, q).all();
            if (find_lane(from, q, all, wave_scan(all))) break;
        }
        __syncthreads();                        // their place is used again
    }
    SequenceWork sw = sequence_work<ROWS>(a, sq);
    int tile = sw.tiles > 1 ? (int)quotient(at - begin, sw.steps) : 0;
    begin += (int64_t)tile * sw.steps;

    while (true) {
        const Unit u = unit_at(a, seq, sq, tile, ROWS);
        const int64_t unit_end = begin + sw.steps, stop = min(unit_end, end);
        const bool starts = at == begin, whole = starts && stop == unit_end;
        // tiles of 16 tokens that this worker has of the unit, and that any row sees
        const int tile_begin = max(sw.tile0 + (int)(at - begin) * (kStep / kTile), u.lo / kTile);
        int tile_end = u.up > u.lo ? (u.up + kTile - 1) / kTile : 0;
        if (!a.whole) tile_end = min(tile_end, sw.tile0 + (int)(stop - begin) * (kStep / kTile));

        v8bf q[RT][2 * J];
        Seen seen[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int row = min(rt * 16 + col, u.rows - 1);
            const uint16_t *from = a.q + row_at(a, u, row, a.ldq, head, D);
#pragma unroll
            for (int k = 0; k < 2 * J; ++k)
                q[rt][k] = query(a, from, k, g);
            seen[rt] = seen_by(a, u.q, (u.row0 + row) / a.group);
        }

        v4f y[RT][DT];
        float m[RT], l[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            m[rt] = -INFINITY;
            l[rt] = 0.0f;
#pragma unroll
            for (int d = 0; d < DT; ++d) y[rt][d] = v4f{0, 0, 0, 0};
        }

        const int tile_shift = c.page_shift - 4;    // tiles of a page, log2
        const int groups = tile_end > tile_begin ? (tile_end - tile_begin + NT - 1) / NT : 0;
        int page = -1;
        float ks = 0.0f, vs = 0.0f;
        int there[NT];                              // pages of the tiles whose codes are on their way
        float kf[NT], vf[NT];
        int64_t tile_at[NT];                        // where they are, in tiles
        // a group's pages: every AHEAD groups a wave looks them up, a tile a lane
        auto find = [&](int gi, int k) {
            if (k % AHEAD == 0) {
                const int tile = tile_begin + (gi + kWaves * (lane / NT)) * NT + lane % NT;
                page = tile < tile_end ? pool_page(c, u.seq, tile >> tile_shift) : -1;
                const int64_t slot = (int64_t)max(page, 0) * c.heads + head;
                ks = c.k_scales[slot];
                vs = c.v_scales[slot];
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                there[t] = __builtin_amdgcn_readlane(page, (k % AHEAD) * NT + t);
                tile_at[t] = (((int64_t)max(there[t], 0) * c.heads + head) << tile_shift) +
                             ((tile_begin + gi * NT + t) & ((1 << tile_shift) - 1));
            }
        };
        auto find_scales = [&](int k) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                kf[t] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ks), (k % AHEAD) * NT + t)) * a.scale;
                vf[t] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(vs), (k % AHEAD) * NT + t));
            }
        };
        uint4 kc[NT][J], vc[NT][J];
        auto load = [&](uint4 (&to)[NT][J], const uint8_t *codes) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const v4u *p = reinterpret_cast<const v4u *>(codes + tile_at[t] * (kTile * D)) + lane;
#pragma unroll
                for (int j = 0; j < J; ++j) to[t][j] = __builtin_bit_cast(uint4, __builtin_nontemporal_load(p + 64 * j));
            }
        };
        if (wave < groups) {
            find(wave, 0);
            load(kc, c.k);
            __builtin_amdgcn_sched_barrier(0);      // in this order the keys can be waited for alone
            load(vc, c.v);
        }
        for (int gi = wave, k = 0; gi < groups; gi += kWaves, ++k) {
            const int tile0 = tile_begin + gi * NT;
            find_scales(k);
            bool edge = tile0 * kTile < u.all_lo || (tile0 + NT) * kTile > u.all_up;
            int mine[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                mine[t] = there[t];
                edge |= mine[t] < 0;
            }
            const bool more = gi + kWaves < groups;
            // scores: row token 4 g + r of tile t, column the lane's query row.  The
            // barriers keep conversions beside the products that take them: hoisted over
            // them, they double the registers.
            v4f x[RT][NT];
#pragma unroll
            for (int t = 0; t < NT; t += 2) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) x[rt][t] = x[rt][t + 1] = v4f{0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < 2 * J; ++k) {
                    const uint4 &c0 = kc[t][k >> 1], &c1 = kc[t + 1][k >> 1];
                    const v8bf k0 = k & 1 ? operand<FMT>(c0.z, c0.w) : operand<FMT>(c0.x, c0.y);
                    const v8bf k1 = k & 1 ? operand<FMT>(c1.z, c1.w) : operand<FMT>(c1.x, c1.y);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        x[rt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, q[rt][k], x[rt][t], 0, 0, 0);
                        x[rt][t + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, q[rt][k], x[rt][t + 1], 0, 0, 0);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            // the next keys, while these scores become probabilities and meet the values
            if (more) {
                find(gi + kWaves, k + 1);
                load(kc, c.k);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (edge) {
                // tokens that no row sees may hold anything: NaN codes must not meet the probability 0
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int token = (tile0 + t) * kTile + 4 * g;
                    uint32_t keep = 0;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const bool any = mine[t] >= 0 && token + r >= u.lo && token + r < u.up;
                        if (any) keep |= 0xFFu << (8 * r);
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt)
                            x[rt][t][r] = any && token + r >= seen[rt].lo && token + r < seen[rt].up ? x[rt][t][r] * kf[t]
                                                                                                     : -INFINITY;
                    }
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        vc[t][j].x &= keep; vc[t][j].y &= keep; vc[t][j].z &= keep; vc[t][j].w &= keep;
                    }
                    kf[t] = 1.0f;
                    if (mine[t] < 0) vf[t] = 0.0f;       // the scale is another page's
                }
            }
            // x kf is the score: the scale of a tile is one for its maximum, and enters each power's argument.
            // The maximum that powers are taken from moves only when a score is 2^8 past it.
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                float top = m[rt];
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    top = fmaxf(top, fmaxf(fmaxf(x[rt][t][0], x[rt][t][1]), fmaxf(x[rt][t][2], x[rt][t][3])) * kf[t]);
                top = row_max(top);
                if (__any(top > m[rt] + 8.0f)) {
                    const float f = top == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m[rt] - top);
                    l[rt] *= f;
#pragma unroll
                    for (int d = 0; d < DT; ++d) y[rt][d] *= f;
                    m[rt] = top;
                }
                const float from = m[rt] == -INFINITY ? 0.0f : m[rt];    // nothing seen yet: all p are 0
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        x[rt][t][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[rt][t][r], kf[t], -from));
                        l[rt] += x[rt][t][r];
                        x[rt][t][r] *= vf[t];
                    }
            }
            __builtin_amdgcn_sched_barrier(0);
            // second product, 32 tokens and 32 channels at a time
#pragma unroll
            for (int t = 0; t < NT; t += 2) {
                v8bf p[RT][TERMS];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) terms<TERMS>(x[rt][t], x[rt][t + 1], p[rt]);
#pragma unroll
                for (int d = 0; d < DT; d += 2) {
                    const uint4 &c0 = vc[t][d >> 2], &c1 = vc[t + 1][d >> 2];
                    const v8bf v0 = d & 2 ? operand<FMT>(c0.z, c1.z) : operand<FMT>(c0.x, c1.x);
                    const v8bf v1 = d & 2 ? operand<FMT>(c0.w, c1.w) : operand<FMT>(c0.y, c1.y);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int n = 0; n < TERMS; ++n) {
                            y[rt][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, p[rt][n], y[rt][d], 0, 0, 0);
                            y[rt][d + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, p[rt][n], y[rt][d + 1], 0, 0, 0);
                        }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            if (more) load(vc, c.v);
        }

        // the waves' sums together, 16 rows at a time
        const int64_t slot = 2 * worker + (starts ? 1 : 0);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            __syncthreads();                        // the last ones are read
            const float sum = row_sum(l[rt]);
            if (g == 0) merge_ml[wave][col] = make_float2(m[rt], sum);
#pragma unroll
            for (int d = 0; d < DT; ++d) *reinterpret_cast<v4f *>(&merge[wave][col][16 * d + 4 * g]) = y[rt][d];
            __syncthreads();
            const int r = threadIdx.x >> 4, row = rt * 16 + r;
            if (row >= u.rows) continue;
            float2 ml[kWaves];
            float top = -INFINITY, total = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                ml[w] = merge_ml[w][r];
                top = fmaxf(top, ml[w].x);
            }
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                ml[w].x = ml[w].x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml[w].x - top);
                total += ml[w].x * ml[w].y;
            }
            const float by = total > 0.0f ? 1.0f / total : 0.0f;
            const int64_t to = row_at(a, u, row, a.ldy, head, D);
#pragma unroll
            for (int k = 0; k < J; ++k) {
                const int d = 64 * k + 4 * (threadIdx.x & 15);
                v4f v = {0, 0, 0, 0};
#pragma unroll
                for (int w = 0; w < kWaves; ++w) v += *reinterpret_cast<const v4f *>(&merge[w][r][d]) * ml[w].x;
                if (whole) store_y4<F32>(a.y, to + d, v * by);
                else *reinterpret_cast<v4f *>(a.part_o + (slot * ROWS + row) * D + d) = v;
            }
            if (!whole && (threadIdx.x & 15) == 0) a.part_ml[slot * ROWS + row] = make_float2(top, total);
        }
        if (stop == end) {
            if (threadIdx.x == 0 && starts && !whole) {      // the unit goes on in other shares
                AttentionCut cut;
                cut.parts = (int)quotient(unit_end - 1, share) - worker + 1;
                cut.place0 = (2 * worker + 1) * ROWS;
                cut.place = 2 * worker * ROWS;
                cut.step = 2 * ROWS;
                cut.head = head;
                cut.first = u.q.first;
                cut.row0 = u.row0;
                cut.rows = u.rows;
                a.cuts[worker] = cut;
            }
            return;
        }
        // the next unit: the sequence's next row tile, the next sequence, the next head
        at = begin = unit_end;
        if (++tile == sw.tiles) {
            tile = 0;
            // 64 at a time: a padded batch may have hundreds without tokens
            for (int from = seq + 1;;) {
                const int s = from + lane;
                Sequence q = {};
                if (s < c.B) q = sequence_at(c, s);
                const uint64_t some = __ballot(sequence_work<ROWS>(a, q).tiles > 0);
                if (some) {
                    const int l = __builtin_ctzll(some);
                    seq = from + l;
                    sq = lane_of(q, l);
                    break;
                }
                from += 64;
                if (from >= c.B) {
                    from = 0;
                    ++head;
                }
            }
            sw = sequence_work<ROWS>(a, sq);
        }
    }
}

// The sums of a unit that was cut.  A workgroup has a row, its parts in sets beside
// each other: 4.6 us for 64 parts of 4 rows (one set after another 13.7), most of it
// three dependent loads.
template <int D, bool F32>
__global__ __launch_bounds__(256) void join_kernel(AttentionLaunch a, const AttentionCut *cuts) {
    constexpr int LANES = D / 4, SETS = 256 / LANES;
    __shared__ float factor[kMostWorkers];
    __shared__ v4f sums[SETS][LANES];
    __shared__ float red[2][4];
    const int row = blockIdx.y, tid = threadIdx.x;
    const AttentionCut cut = cuts[blockIdx.x];
    if (cut.parts <= 1 || row >= cut.rows) return;
    const int parts = cut.parts;
    auto place = [&](int p) { return (int64_t)(p == 0 ? cut.place0 : cut.place + p * cut.step) + row; };
    float top = -INFINITY;
    for (int p = tid; p < parts; p += 256) top = fmaxf(top, a.part_ml[place(p)].x);
    top = wave_max(top);
    if ((tid & 63) == 0) red[0][tid >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    float total = 0.0f;
    for (int p = tid; p < parts; p += 256) {
        const float2 ml = a.part_ml[place(p)];
        const float f = ml.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml.x - top);
        factor[p] = f;
        total += f * ml.y;
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) total += __shfl_xor(total, d);
    if ((tid & 63) == 0) red[1][tid >> 6] = total;
    __syncthreads();
    total = red[1][0] + red[1][1] + red[1][2] + red[1][3];
    const int set = tid / LANES, lane = tid % LANES;
    if (set < SETS) {
        v4f v = {0, 0, 0, 0};
#pragma unroll 4
        for (int p = set; p < parts; p += SETS)
            v += *reinterpret_cast<const v4f *>(a.part_o + place(p) * D + 4 * lane) * factor[p];
        sums[set][lane] = v;
    }
    __syncthreads();
    if (tid < LANES) {
        v4f v = sums[0][tid];
#pragma unroll
        for (int s = 1; s < SETS; ++s) v += sums[s][tid];
        const int at = cut.row0 + row, token = at / a.group;
        store_y4<F32>(a.y,
                      (int64_t)(cut.first + token) * a.ldy + (int64_t)(cut.head * a.group + at - token * a.group) * D + 4 * tid,
                      v * (total > 0.0f ? 1.0f / total : 0.0f));
    }
}

template <int D, int FMT, int TERMS, int RT>
void launch_rows(const AttentionLaunch &a, hipStream_t s) {
    hipLaunchKernelGGL((attention_kernel<D, FMT, TERMS, RT>), dim3(a.workers), dim3(64 * kWaves), 0, s, a);
}

template <int D, int FMT>
void launch_width(bool f32, const AttentionPlan &p, const AttentionLaunch &a, hipStream_t s) {
    if (p.workers > 0) {
        if (p.rows == 16) f32 ? launch_rows<D, FMT, 3, 1>(a, s) : launch_rows<D, FMT, 2, 1>(a, s);
        else f32 ? launch_rows<D, FMT, 3, 2>(a, s) : launch_rows<D, FMT, 2, 2>(a, s);
    }
    if (p.wide_units > 0) launch_wide(FMT, f32, D, a, s);
    auto join = [&](const AttentionCut *cuts, int64_t entries, int rows) {
        if (f32) hipLaunchKernelGGL((join_kernel<D, true>), dim3(entries, rows), dim3(256), 0, s, a, cuts);
        else hipLaunchKernelGGL((join_kernel<D, false>), dim3(entries, rows), dim3(256), 0, s, a, cuts);
    };
    if (p.workers > 1 && !p.whole) join(a.cuts, p.workers - 1, p.live_rows);
    if (p.wide_parts > 1) join(a.wide_cuts, p.wide_units, p.wide_rows);
}

template <int FMT>
void launch_format(bool f32, int head_dim, const AttentionPlan &p, const AttentionLaunch &a, hipStream_t s) {
    switch (head_dim) {
    case 64: launch_width<64, FMT>(f32, p, a, s); break;
    case 128: launch_width<128, FMT>(f32, p, a, s); break;
    case 192: launch_width<192, FMT>(f32, p, a, s); break;
    default: launch_width<256, FMT>(f32, p, a, s); break;
    }
}

// row tiles of a key head: each sequence with n tokens has ceil(n group / rows)
int64_t row_tiles(int64_t sequences, int64_t tokens, int group, int rows) {
    const int64_t some = std::min(sequences, tokens);
    return std::min((tokens * group + some * (rows - 1)) / rows, tokens * ((group + rows - 1) / rows));
}

constexpr int kWideItems = 512;    // (unit, head, part) workgroups that wide units are split for
constexpr int kWideChunk = 256;    // expected tokens of a part, at least

// Parts of a wide unit: the time of a part's steps, 1.5 us each or 2.4 where two workgroups share a
// compute unit, and of the join: a launch, and partial sums written and read at 4 TB/s.  512 tokens alone
// (32 / 8 heads of 128) take 21.9 us with one part and 32.9 with two; 512 after 3600, 73 with four and 81
// with two; 64 over 8000, 29.0 with 16, 31.4 with 32 and 40.6 with eight; 100 over 2000 (heads of 64),
// 19.0 with eight and 23.8 with four.  (Steps are 1.7 and 3.0 us with two terms; chosen by those, 192 rows
// alone over 30000 tokens take 66 us for 58, 512 rows 105 for 112, and most calls the same.)
int wide_parts(int64_t units, int64_t most, int max_context, int head_dim) {
    const double steps = max_context / (head_dim <= 128 ? 64.0 : 32.0);
    const double sums = units * wide_rows(head_dim) * head_dim * 8 / 4e6;
    int best = 1;
    double least = 0.0;
    for (int64_t parts = 1; parts <= std::max<int64_t>(1, std::min(kWideItems / units, most)); ++parts) {
        const double us = steps / parts * (units * parts > 256 ? 2.4 : 1.5) + (parts > 1 ? 5.0 + sums * parts : 0.0);
        if (parts > 1 && us >= least) continue;
        least = us;
        best = (int)parts;
    }
    return best;
}

}  // namespace

AttentionPlan attention_plan(int sequences, int tokens, int max_context, int kv_heads, int group, int head_dim) {
    AttentionPlan p = {};
    if (sequences == 0 || tokens == 0) return p;
    const int64_t all_rows = (int64_t)tokens * group;
    const int64_t steps = ((int64_t)max_context + kStep - 1) / kStep + 1;
    // a unit of so few tokens is read as fast by one workgroup as cut and joined (see above)
    const int whole = head_dim <= 128 ? 4 * kStep : 2 * kStep;

    // Which sequences have few rows is known on the device alone: of several, some may
    // have few and some many, and both kernels run, each with its own.
    const bool wide = sequences == 1 ? all_rows >= kWideFromAlone
                                     : (tokens - std::min(sequences, tokens)) * (int64_t)group >= kWideFrom;
    const bool few = !wide || sequences > 1;
    p.few_rows = !wide ? INT32_MAX : few ? few_rows(head_dim) : 0;
    if (few) {
        // 16 rows in a unit, or 32: as a sequence has on average.  An average beyond this kernel's sequences says that
        // some have many rows, and then 16 for the others, single tokens for the most part.  Between 16 and that it is
        // drafts (4 tokens of 64 sequences of 4096, 8 query heads a key head: 98 us with 32 rows, 175 with 16, which read all
        // codes twice), or single tokens beside a prompt that draws the average up, which lose less (400 tokens beside 63
        // single ones over 2000, 4 query heads a key head: 112.6 with 32 rows, 109 with 16; 1000 of 128 over 1000: 92.6 and 87.5).
        const bool prompts = wide && all_rows > few_rows(head_dim) * (int64_t)sequences;
        p.rows = all_rows <= 16 * (int64_t)sequences || (prompts && group <= 16) ? 16 : 32;
        p.live_rows = (int)std::min<int64_t>(p.rows, all_rows);
        const int64_t units = row_tiles(sequences, tokens, group, p.rows) * kv_heads;
        p.whole = max_context <= whole;
        // As many workers as are resident at once.  (Registers: 122 for heads of 64, 161 of 128, up to 241 of 256;
        // of 32 rows 204, 256, and over 256 for wider heads.)  With fewer, ragged lengths take longer, 64
        // contexts of up to 8192 for heads of 64 42.9 us with 512 and 40.4 with 768; with more, they wait.
        const int64_t most = 256 * (p.rows == 32 && head_dim > 128 ? 1 : head_dim == 64 && p.rows == 16 ? 3 : 2);
        p.workers = (int)(p.whole ? std::min<int64_t>(units, kMostWorkers) : std::min(most, units * steps));
    }
    if (wide) {
        p.wide_rows = wide_rows(head_dim);
        p.wide_units = row_tiles(sequences, tokens, group, p.wide_rows) * kv_heads;
        p.wide_parts = wide_parts(p.wide_units, (max_context + kWideChunk - 1) / kWideChunk, max_context, head_dim);
    }
    // The workspace of any plan of as many or fewer sequences, tokens and context
    if (max_context > std::min(whole, kWideChunk)) {      // else no unit is cut
        const int64_t few_most = std::min<int64_t>(kMostWorkers, row_tiles(sequences, tokens, group, 16) * kv_heads * steps);
        const int64_t slots = few_most * 2 * (all_rows <= 16 ? 16 : 32);
        const int64_t wide_most = std::min<int64_t>(kWideItems, row_tiles(sequences, tokens, group, 64) * kv_heads *
                                                                    ((max_context + kWideChunk - 1) / kWideChunk));
        const int64_t wide_slots = all_rows >= kWideFromAlone ? wide_most * 128 : 0;
        p.wide_place = slots;
        p.ml_at = (size_t)(slots + wide_slots) * head_dim * sizeof(float);
        p.cuts_at = p.ml_at + (size_t)(slots + wide_slots) * sizeof(float2);
        p.wide_cuts_at = p.cuts_at + (size_t)few_most * sizeof(AttentionCut);
        p.ws_bytes = p.wide_cuts_at + (wide_slots ? (size_t)wide_most * sizeof(AttentionCut) : 0);
    }
    return p;
}

hipError_t launch_attention(int fmt, bool f32, int head_dim, const AttentionPlan &p, const AttentionLaunch &a,
                            hipStream_t s) {
    if (fmt == FMT_I8) launch_format<FMT_I8>(f32, head_dim, p, a, s);
    else launch_format<FMT_FP8>(f32, head_dim, p, a, s);
    return hipGetLastError();
}

}  // namespace qlin
