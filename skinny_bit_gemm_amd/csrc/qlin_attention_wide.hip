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
// Where y is bf16, probabilities enter the second product as one fp16 number (11
// bits of mantissa, 2^-11 against 2^-8 of y's own rounding), and codes as fp16, which
// holds them exactly.  The scales of the values would leave its range, so they enter
// relative to a power of two that the sums are kept in, and that follows the scales
// (Base).  Where y is fp32: three bf16 terms, 24 bits.
//
// 3558 tokens of three prompts over up to 8192, 32 query heads over 8 of 128, e4m3, y
// bf16 (370 GFLOP): 498 us, 740 TFLOP/s.  Of a step's 6800 cycles for the two waves of a
// SIMD the matrix cores work 2050 (32 and 32 products a wave), the vector ALUs some 3200
// (300 instructions and 34 powers a wave), the LDS 2560; with two waves what is left
// are the waits between them.  Without conversions it takes 425 us, without powers 35
// less, without either product about as long.  Measured and slower: 16 rows a wave and
// eight waves (674), eight waves of 32 rows (545), steps of 32 tokens (604; with three
// waves a SIMD 734, spilled), the two tiles of rows one behind the other so that
// powers and products share a stretch (740: each reads the LDS for itself, and
// spills), 635 with maxima that move each time and a branch for each tile's edge and scale.
#include "qlin_attention.h"

namespace qlin {

namespace {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// four codes of a word as fp16 (exact)
template <int FMT>
__device__ __forceinline__ uint2 f16_codes(uint32_t w) {
    if constexpr (FMT == FMT_I8) {
        // 1024 + (code + 128) is the fp16 number 0x6400 + code + 128
        const uint32_t u = w ^ 0x80808080u;
        const v2h off = {(_Float16)1152.0f, (_Float16)1152.0f};
        const v2h lo = __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) - off;
        const v2h hi = __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) - off;
        return make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
    }
    return make_uint2(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true)));
}

// exponent of a scale's power of two, in fp32's bias; of those too small for it, the lowest
__device__ __forceinline__ int exponent(float v) { return max((int)(__float_as_uint(v) >> 23 & 0xFFu), 1); }

template <int D, int FMT, bool F32, int RT>
__global__ __launch_bounds__(64 * kWaves, 2) void wide_kernel(AttentionLaunch a) {
    constexpr int WROWS = 16 * RT, ROWS = kWaves * WROWS, J = D / 64, DT = D / 16, NT = D <= 128 ? 4 : 2;
    constexpr int AHEAD = 64 / NT, TERMS = F32 ? 3 : 1;
    constexpr int KU = (NT * J + kWaves - 1) / kWaves, VU = (NT / 2 * J + kWaves - 1) / kWaves;   // a wave's pieces of a step
    __shared__ v4u keys[2][NT * 2 * J][64];
    __shared__ v4u values[2][NT / 2 * DT][64];
    const CacheArgs &c = a.c;
    const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tile_shift = c.page_shift - 4;

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
        float ks, vs;
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
                const int t = min(wave + kWaves * i, NT / 2 * J - 1) % (NT / 2) * 2 + h, token = (tile0 + t) * kTile + 4 * g;
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
            for (int d = 0; d < 4; ++d) {
                v4u w;
                if constexpr (F32) {
                    w = __builtin_bit_cast(v4u, operand<FMT>(w0[d], w1[d]));
                } else {
                    const uint2 lo = f16_codes<FMT>(w0[d]), hi = f16_codes<FMT>(w1[d]);
                    w = v4u{lo.x, lo.y, hi.x, hi.y};
                }
                values[b][t * DT + 4 * j + d][lane] = w;
            }
        }
    };

    // Base: a scale over 2^(base - 127) is between 2^-4 and 2^5, so a probability below fp16's
    // normal numbers is off by 2^-21 of its value's magnitude at most.
    int base = 0;                               // y's sums are times 2^(127 - base)
    float weight = 0.0f;                        // a tile's scale in them
    uint64_t valued = 0, plain = 0;             // lanes whose tiles have a scale that is not 0, and one near base
    auto set_base = [&](int to) {
        base = to;
        weight = F32 ? now.vs : __builtin_ldexpf(now.vs, 127 - base);
        valued = __ballot(now.vs != 0.0f);
        plain = valued & __ballot((unsigned)(exponent(now.vs) - (base - 4)) <= 8u);
    };
    auto rebase = [&](int to) {
        const int next_base = max(to, base - 80);       // sums of 2^30 tokens stay in fp32
        const float f = __builtin_ldexpf(1.0f, max(base - next_base, -126));
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int d = 0; d < DT; ++d) y[rt][d] *= f;
        set_base(next_base);
    };
    auto value = [&](int b, int t, int d) { return __builtin_bit_cast(v8h, values[b][t / 2 * DT + d][lane]); };
    // y += V^T P^T of tiles t and t + 1, their probabilities times f0 and f1
    auto multiply = [&](int b, int t, const v4f (&x)[RT][NT], float f0, float f1) {
        if constexpr (F32) {
            v8bf p[RT][TERMS];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) terms<TERMS>(x[rt][t] * f0, x[rt][t + 1] * f1, p[rt]);
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const v8bf v = __builtin_bit_cast(v8bf, value(b, t, d));
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int n = 0; n < TERMS; ++n)
                        y[rt][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p[rt][n], y[rt][d], 0, 0, 0);
            }
        } else {
            v8h p[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p[rt][i] = (_Float16)(x[rt][t][i] * f0);
                    p[rt][4 + i] = (_Float16)(x[rt][t + 1][i] * f1);
                }
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const v8h v = value(b, t, d);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
                    y[rt][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, p[rt], y[rt][d], 0, 0, 0);
            }
        }
    };

    __syncthreads();                            // the buffers may still be read for the item before
    if (groups > 0) {
        load(0);
        hide(0);
        convert(0);
        now = next;
        set_base(base);
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
        if (gi + 2 < groups) load(gi + 2);
        if (needed) {
            float kf[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) kf[t] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(now.ks), lane0 + t));
            if (edge) {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int token = (tile0 + t) * kTile + 4 * g;
                    const bool there = now.there >> (lane0 + t) & 1;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt)
                            x[rt][t][r] = there && token + r >= seen[rt].lo && token + r < seen[rt].up ? x[rt][t][r] * kf[t]
                                                                                                       : -INFINITY;
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
                for (int t = 0; t < NT; ++t)
                    top[rt] = fmaxf(top[rt], fmaxf(fmaxf(x[rt][t][0], x[rt][t][1]), fmaxf(x[rt][t][2], x[rt][t][3])) * kf[t]);
                top[rt] = row_max(top[rt]);
                moves |= top[rt] > m[rt] + 8.0f;
            }
            if (__any(moves)) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const float f = top[rt] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m[rt] - top[rt]);
                    l[rt] *= f;
#pragma unroll
                    for (int d = 0; d < DT; ++d) y[rt][d] *= f;
                    m[rt] = top[rt];
                }
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const float from = m[rt] == -INFINITY ? 0.0f : m[rt];        // nothing seen yet: all p are 0
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        x[rt][t][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[rt][t][r], kf[t], -from));
                        l[rt] += x[rt][t][r];
                    }
            }
            // The tiles whose scales are near base, which is nearly always all of them; then, for what is
            // left, a base near the first of it.
            uint64_t left = F32 ? STEP : valued >> lane0 & STEP;
            while (left) {
                if (!F32 && (plain >> lane0 & left) == 0)
                    rebase(exponent(__uint_as_float(
                        __builtin_amdgcn_readlane(__float_as_uint(now.vs), lane0 + __builtin_ctzll(left)))));
                const uint64_t mine = F32 ? STEP : plain >> lane0 & left;
                float f[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint32_t w = __builtin_amdgcn_readlane(__float_as_uint(weight), lane0 + t);
                    f[t] = __uint_as_float(mine >> t & 1 ? w : 0u);
                }
#pragma unroll
                for (int t = 0; t < NT; t += 2) multiply(b, t, x, f[t], f[t + 1]);
                left &= ~mine;
            }
        }
        if ((gi + 1) % AHEAD == 0) {
            now = next;
            set_base(base);
        }
        __syncthreads();
    }

    const float unit_of_y = F32 ? 1.0f : __builtin_ldexpf(1.0f, base - 127);
    const int64_t first_place = a.wide_place + (place * a.wide_parts + part) * ROWS;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const float total = row_sum(l[rt]);
        const int row = wrow0 + rt * 16 + col;
        if (row >= u.rows) continue;
        if (a.wide_parts > 1) {
#pragma unroll
            for (int d = 0; d < DT; ++d)
                *reinterpret_cast<v4f *>(a.part_o + (first_place + row) * D + 16 * d + 4 * g) = y[rt][d] * unit_of_y;
            if (g == 0) a.part_ml[first_place + row] = make_float2(m[rt], total);
        } else {
            const float by = total > 0.0f ? unit_of_y / total : 0.0f;
            const int64_t to = row_at(a, u, row, a.ldy, head, D);
#pragma unroll
            for (int d = 0; d < DT; ++d) store_y4<F32>(a.y, to + 16 * d + 4 * g, y[rt][d] * by);
        }
    }
    if (a.wide_parts > 1 && part == 0 && threadIdx.x == 0) {
        AttentionCut cut;
        cut.parts = a.wide_parts;
        cut.place0 = cut.place = (int)first_place;
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
