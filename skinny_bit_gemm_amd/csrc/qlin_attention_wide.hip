// qlin_attention_wide.hip -- attention over the paged 8-bit cache for sequences
// with many query rows (pieces of prompts): bound by the matrix cores and by the
// vector instructions of the softmax.
//
// A workgroup has 64 RT rows, 16 RT for each wave, and goes over its tokens in
// steps of NT tiles of 16.  The codes of a step are read and converted once for the
// four waves, into the LDS in the operands' order (each read of a wave is 1 KiB of
// consecutive bytes); two buffers, so that the next step is converted while this one
// is multiplied, and the one behind it is on its way from memory.
//
// Probabilities, times their page's scale, enter the second product as two bf16 terms where y
// is bf16 (16 bits of mantissa) and three where it is fp32 (24), as in the kernel for few rows, so
// that a query's result is as exact however many rows its sequence brings.  One fp16 number (11
// bits, and fewer below its normal range: a first token with nearly all the weight and a value of 0
// leaves the others there, and the scales of a unit's pages have to fit its range) takes 424 us
// where this takes 530.
//
// 3558 tokens of three prompts over up to 8192, 32 query heads over 8 of 128, e4m3, y
// bf16 (370 GFLOP): 530 us, 700 TFLOP/s; y fp32: 662 us, 560 TFLOP/s.  The powers of two tiles are
// computed beside the products of the two before, whose operands are read from the LDS a while
// before.  Two waves a SIMD.  Chosen while probabilities were one fp16 number, by us of the same
// call: where it took 500, all powers first 499, reads next to their products 491, both as
// now 442; 16 rows a wave and eight waves 674, eight waves of 32 rows 545, steps of 32 tokens
// 604 (with three waves a SIMD 734, spilled), the two tiles of rows one behind the other 740
// (each reads the LDS for itself, and spills), maxima that move each time and a branch for each
// tile's edge and scale 635, waves of a higher priority in the products 523; where it took
// 424, a barrier in the middle of a step with three buffers of values 433, four or twelve
// reads of values ahead 440, 443.  With two terms, the order of the terms' products and a first
// term that is cut instead of rounded change nothing (526 each).
//
// Built with -fno-honor-nans, without which each fmaxf quiets its operands first (436 us
// where it was 424, 24 of 267 instructions of a step): what may be NaN in hidden places is
// replaced as bits.
#include "qlin_attention.h"

namespace qlin {

namespace {

// A step's tiles, and its operands in the LDS.
constexpr int tiles_of_step(int D) { return D <= 128 ? 4 : 2; }

template <int D>
struct Operands {
    v4u keys[2][tiles_of_step(D) * (D / 32)][64];
    v4u values[2][tiles_of_step(D) / 2 * (D / 16)][64];
};

// A part of a unit: what its tokens of tiles tile_begin to tile_end add.
template <int D, int FMT, bool F32, int RT>
__device__ __forceinline__ void unit_part(const AttentionLaunch &a, Operands<D> &sh, const Unit &u, int seq, int head,
                                          int tile_begin, int tile_end, int64_t place, int part) {
    constexpr int WROWS = 16 * RT, ROWS = kWaves * WROWS, J = D / 64, DT = D / 16, NT = tiles_of_step(D);
    constexpr int TERMS = F32 ? 3 : 2;          // of a probability
    constexpr int AHEAD = 64 / NT;
    constexpr int PRE = NT / 2 * DT < 8 ? NT / 2 * DT : 8;
    // a wave's pieces of a step
    constexpr int KU = (NT * J + kWaves - 1) / kWaves, VU = (NT / 2 * J + kWaves - 1) / kWaves;
    auto &keys = sh.keys;
    auto &values = sh.values;
    const CacheArgs &c = a.c;
    const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tile_shift = c.page_shift - 4;
    const int groups = tile_end > tile_begin ? (tile_end - tile_begin + NT - 1) / NT : 0;

    // this wave's rows, and what they see
    const int wrow0 = wave * WROWS, wrows = min(WROWS, u.rows - wrow0);
    v8bf q[RT][2 * J];
    Seen seen[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int row = min(wrow0 + rt * 16 + col, u.rows - 1);
        const uint16_t *from = a.q + row_at(a, u, row, a.ldq, head, D);
#pragma unroll
        for (int k = 0; k < 2 * J; ++k) q[rt][k] = query(a, from, k, g);
        seen[rt] = seen_by(a, u.q, (u.row0 + row) / a.group);
    }
    Seen any = {0, 0}, all = {0, 0};
    if (wrows > 0) {
        const Seen first = seen_by(a, u.q, (u.row0 + wrow0) / a.group);
        const Seen last = seen_by(a, u.q, (u.row0 + wrow0 + wrows - 1) / a.group);
        any = {first.lo, last.up};
        all = {last.lo, first.up};
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

    // Pages and scales of AHEAD steps, a tile a lane: of the steps whose codes are on their way, and of
    // those that are multiplied.
    struct Pages {
        int64_t at;                             // where the tile's codes are
        uint64_t there;                         // lanes whose page is
        float ks, vs;                           // scales of keys, times the scores', and of values
    };
    Pages next = {0, 0, 0, 0}, now = next;
    auto look_up = [&](int gi) {
        const int tile = tile_begin + gi * NT + lane;
        const int page = tile < tile_end ? pool_page(c, seq, tile >> tile_shift) : -1;
        const int64_t slot = (int64_t)max(page, 0) * c.heads + head;
        next.there = __ballot(page >= 0);
        next.ks = c.k_scales[slot] * a.scale;
        next.vs = page >= 0 ? c.v_scales[slot] : 0.0f;
        next.at = ((slot << tile_shift) + (tile & ((1 << tile_shift) - 1))) * (kTile * D);
    };
    auto lane_of = [&](int gi) { return gi % AHEAD * NT; };
    uint4 kc[KU], vc[VU][2];
    auto load = [&](int gi) {                   // a step's codes, this wave's pieces
        if (gi % AHEAD == 0) look_up(gi);
        auto at = [&](const uint8_t *codes, int t, int j) {
            const int lo = __builtin_amdgcn_readlane((int)next.at, lane_of(gi) + t);
            const int hi = __builtin_amdgcn_readlane((int)(next.at >> 32), lane_of(gi) + t);
            const int64_t tile = (int64_t)((uint64_t)(uint32_t)hi << 32 | (uint32_t)lo);
            return *(reinterpret_cast<const uint4 *>(codes + tile + 1024 * j) + lane);
        };
#pragma unroll
        for (int i = 0; i < KU; ++i) {
            const int piece = min(wave + kWaves * i, NT * J - 1);
            kc[i] = at(c.k, piece % NT, piece / NT);
        }
#pragma unroll
        for (int i = 0; i < VU; ++i) {
            const int piece = min(wave + kWaves * i, NT / 2 * J - 1);
            vc[i][0] = at(c.v, piece % (NT / 2) * 2, piece / (NT / 2));
            vc[i][1] = at(c.v, piece % (NT / 2) * 2 + 1, piece / (NT / 2));
        }
    };
    constexpr uint64_t STEP = (1ull << NT) - 1;
    auto pages_there = [&](const Pages &p, int gi) { return (p.there >> lane_of(gi) & STEP) == STEP; };
    // Tokens that no row sees may hold anything: NaN codes must not meet the probability 0.
    auto hide = [&](int gi) {
        const int tile0 = tile_begin + gi * NT;
        if (pages_there(next, gi) && tile0 * kTile >= u.lo && (tile0 + NT) * kTile <= u.up) return;
#pragma unroll
        for (int i = 0; i < VU; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = min(wave + kWaves * i, NT / 2 * J - 1) % (NT / 2) * 2 + h;
                const int token = (tile0 + t) * kTile + 4 * g;
                const bool there = next.there >> (lane_of(gi) + t) & 1;
                uint32_t keep = 0;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (there && token + r >= u.lo && token + r < u.up) keep |= 0xFFu << (8 * r);
                vc[i][h].x &= keep; vc[i][h].y &= keep; vc[i][h].z &= keep; vc[i][h].w &= keep;
            }
    };
    // What load() brought, as operands, into the buffer of step gi.  (A wave without a piece of
    // its own repeats the last one.)
    auto convert = [&](int gi) {
        const int b = gi & 1;
#pragma unroll
        for (int i = 0; i < KU; ++i) {
            const int piece = min(wave + kWaves * i, NT * J - 1), t = piece % NT, j = piece / NT;
            keys[b][t * 2 * J + 2 * j][lane] = __builtin_bit_cast(v4u, operand<FMT>(kc[i].x, kc[i].y));
            keys[b][t * 2 * J + 2 * j + 1][lane] = __builtin_bit_cast(v4u, operand<FMT>(kc[i].z, kc[i].w));
        }
#pragma unroll
        for (int i = 0; i < VU; ++i) {
            const int piece = min(wave + kWaves * i, NT / 2 * J - 1), t = piece % (NT / 2), j = piece / (NT / 2);
            const uint32_t w0[4] = {vc[i][0].x, vc[i][0].y, vc[i][0].z, vc[i][0].w};
            const uint32_t w1[4] = {vc[i][1].x, vc[i][1].y, vc[i][1].z, vc[i][1].w};
#pragma unroll
            for (int d = 0; d < 4; ++d)
                values[b][t * DT + 4 * j + d][lane] = __builtin_bit_cast(v4u, operand<FMT>(w0[d], w1[d]));
        }
    };

    // y += V^T P^T of tiles t and t + 1, their probabilities times f0 and f1
    auto multiply = [&](int t, const v4f (&x)[RT][NT], float f0, float f1, auto &&value) {
        v8bf p[RT][TERMS];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) terms<TERMS>(x[rt][t] * f0, x[rt][t + 1] * f1, p[rt]);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            const v8bf v = __builtin_bit_cast(v8bf, value(d));
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int n = 0; n < TERMS; ++n)
                    y[rt][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p[rt][n], y[rt][d], 0, 0, 0);
        }
    };

    __syncthreads();                            // the buffers may still be read for the item before
    if (groups > 0) {
        load(0);
        hide(0);
        convert(0);
        now = next;
    }
    if (groups > 1) load(1);
    __syncthreads();
    for (int gi = 0; gi < groups; ++gi) {
        const int b = gi & 1, tile0 = tile_begin + gi * NT, lane0 = lane_of(gi);
        const bool needed = tile0 * kTile < any.up && (tile0 + NT) * kTile > any.lo;
        const bool edge = tile0 * kTile < all.lo || (tile0 + NT) * kTile > all.up || !pages_there(now, gi);
        v4f x[RT][NT];
        if (gi + 1 < groups) hide(gi + 1);
        // Scores: row token 4 g + r of tile t, column the lane's query row.  The next channels'
        // operands are on their way from the LDS while these are multiplied, and the next step's
        // codes are converted beside the products.
        {
            v8bf kk[2][NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                kk[0][t] = __builtin_bit_cast(v8bf, keys[b][t * 2 * J][lane]);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) x[rt][t] = v4f{0, 0, 0, 0};
            }
#pragma unroll
            for (int k = 0; k < 2 * J; ++k) {
                if (k + 1 < 2 * J) {
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        kk[(k + 1) & 1][t] = __builtin_bit_cast(v8bf, keys[b][t * 2 * J + k + 1][lane]);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
                        x[rt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kk[k & 1][t], q[rt][k], x[rt][t], 0, 0, 0);
            }
            convert(gi + 1);                    // past the last step: what was there, into the free buffer
        }
        if (needed) {
            // the first values, a while before they are multiplied
            v4u ready[PRE];
#pragma unroll
            for (int i = 0; i < PRE; ++i) ready[i] = values[b][i][lane];
            float kf[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t)
                kf[t] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(now.ks), lane0 + t));
            if (__builtin_expect(edge, 0)) {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int token = (tile0 + t) * kTile + 4 * g;
                    const bool there = now.there >> (lane0 + t) & 1;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) {
                            const bool sees = there && token + r >= seen[rt].lo && token + r < seen[rt].up;
                            const uint32_t score = __float_as_uint(x[rt][t][r] * kf[t]);
                            x[rt][t][r] = __uint_as_float(sees ? score : 0xFF800000u);
                        }
                    kf[t] = 1.0f;
                }
            }
            // x kf is the score: the scale of a tile is one for its maximum, and enters each power's argument.
            // The maximum that powers are taken from moves only when a score is 2^8 past it.
            float top[RT];
            bool moves = false;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                top[rt] = m[rt];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const v4f &s = x[rt][t];
                    top[rt] = fmaxf(top[rt], fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])) * kf[t]);
                }
                top[rt] = row_max(top[rt]);
                moves |= top[rt] > m[rt] + 8.0f;
            }
            if (__builtin_expect(__any(moves), 0)) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const float f = top[rt] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m[rt] - top[rt]);
                    l[rt] *= f;
#pragma unroll
                    for (int d = 0; d < DT; ++d) y[rt][d] *= f;
                    m[rt] = top[rt];
                }
            }
            float from[RT];                         // where nothing is seen yet, all p are 0
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) from[rt] = m[rt] == -INFINITY ? 0.0f : m[rt];
            auto powers = [&](int t) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float p = x[rt][t + i / 4][i % 4];
                        x[rt][t + i / 4][i % 4] = __builtin_amdgcn_exp2f(__builtin_fmaf(p, kf[t + i / 4], -from[rt]));
                    }
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const v4f s = x[rt][t] + x[rt][t + 1];
                    l[rt] += (s[0] + s[1]) + (s[2] + s[3]);
                }
            };
            auto vs_of = [&](int t) {
                return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(now.vs), lane0 + t));
            };
            // powers of two tiles beside the products of the two before
#pragma unroll
            for (int t = 0; t < NT; t += 2) {
                powers(t);
                multiply(t, x, vs_of(t), vs_of(t + 1), [&](int d) {
                    const int piece = t / 2 * DT + d;
                    const v4u v = ready[piece % PRE];
                    if (piece + PRE < NT / 2 * DT) ready[piece % PRE] = values[b][piece + PRE][lane];
                    return v;
                });
            }
        }
        if (gi + 2 < groups) load(gi + 2);
        if ((gi + 1) % AHEAD == 0) now = next;
        __syncthreads();
    }

    const int64_t first_place = a.wide_place + (place * a.wide_parts + part) * ROWS;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const float total = row_sum(l[rt]);
        const int row = wrow0 + rt * 16 + col;
        if (row >= u.rows) continue;
        if (a.wide_parts > 1) {
#pragma unroll
            for (int d = 0; d < DT; ++d)
                *reinterpret_cast<v4f *>(a.part_o + (first_place + row) * D + 16 * d + 4 * g) = y[rt][d];
            if (g == 0) a.part_ml[first_place + row] = make_float2(m[rt], total);
        } else {
            const float by = total > 0.0f ? 1.0f / total : 0.0f;
            const int64_t to = row_at(a, u, row, a.ldy, head, D);
#pragma unroll
            for (int d = 0; d < DT; ++d) store_y4<F32>(a.y, to + 16 * d + 4 * g, y[rt][d] * by);
        }
    }
}

template <int D, int FMT, bool F32, int RT>
__global__ __launch_bounds__(64 * kWaves, 2) void wide_kernel(AttentionLaunch a) {
    constexpr int ROWS = kWaves * 16 * RT, NT = tiles_of_step(D);
    __shared__ Operands<D> sh;
    const CacheArgs &c = a.c;

    const int64_t items = a.wide_units * a.wide_parts;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int part = (int)(item / a.wide_units);
        const int64_t place = item - part * a.wide_units;       // (unit, head): heads beside each other
        const int unit = (int)(place / c.heads), head = (int)(place - (int64_t)unit * c.heads);
        int within;
        auto tiles_of = [&](const Sequence &q) {
            return (int64_t)q.n * a.group > a.few_rows ? (q.n * a.group + ROWS - 1) / ROWS : 0;
        };
        const int seq = unit_sequence(c, unit, tiles_of, &within);
        if (seq < 0) {
            if (a.wide_parts > 1 && part == 0 && threadIdx.x == 0) a.wide_cuts[place].parts = 0;
            continue;
        }
        const Sequence sq = sequence_at(c, seq);
        // the last rows first: of a prompt, they see the most
        const Unit u = unit_at(a, seq, sq, tiles_of(sq) - 1 - within, ROWS);
        int tile_begin = u.lo / kTile, tile_end = u.up > u.lo ? (u.up + kTile - 1) / kTile : tile_begin;
        if (a.wide_parts > 1) {
            // whole steps of the unit's tokens in each part
            const int steps = (tile_end - tile_begin + NT - 1) / NT, from = tile_begin, all = tile_end;
            tile_begin = from + (int)((int64_t)steps * part / a.wide_parts) * NT;
            tile_end = min(all, from + (int)((int64_t)steps * (part + 1) / a.wide_parts) * NT);
        }

        unit_part<D, FMT, F32, RT>(a, sh, u, seq, head, tile_begin, tile_end, place, part);
        if (a.wide_parts > 1 && part == 0 && threadIdx.x == 0) {
            AttentionCut cut;
            cut.parts = a.wide_parts;
            cut.place0 = cut.place = (int)(a.wide_place + place * a.wide_parts * ROWS);
            cut.step = ROWS;
            cut.head = head;
            cut.first = u.q.first;
            cut.row0 = u.row0;
            cut.rows = u.rows;
            a.wide_cuts[place] = cut;
        }
    }
}

template <int D, int RT>
void launch_types(int fmt, bool f32, const AttentionLaunch &a, hipStream_t s) {
    const int64_t items = a.wide_units * a.wide_parts;
    const dim3 grid((unsigned)(items < 1 << 20 ? items : 1 << 20)), block(64 * kWaves);
    if (fmt == FMT_I8) {
        if (f32) hipLaunchKernelGGL((wide_kernel<D, FMT_I8, true, RT>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((wide_kernel<D, FMT_I8, false, RT>), grid, block, 0, s, a);
    } else {
        if (f32) hipLaunchKernelGGL((wide_kernel<D, FMT_FP8, true, RT>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((wide_kernel<D, FMT_FP8, false, RT>), grid, block, 0, s, a);
    }
}

}  // namespace

void launch_wide(int fmt, bool f32, int head_dim, const AttentionLaunch &a, hipStream_t s) {
    switch (head_dim) {
    case 64: launch_types<64, 2>(fmt, f32, a, s); break;
    case 128: launch_types<128, 2>(fmt, f32, a, s); break;
    case 192: launch_types<192, 2>(fmt, f32, a, s); break;
    default: launch_types<256, 1>(fmt, f32, a, s); break;
    }
}

}  // namespace qlin
