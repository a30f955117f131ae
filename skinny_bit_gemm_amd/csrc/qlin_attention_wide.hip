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
    int base = 0;                               // y's sums are times 2^(127 - base)
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        m[rt] = -INFINITY;
        l[rt] = 0.0f;
#pragma unroll
        for (int d = 0; d < DT; ++d) y[rt][d] = v4f{0, 0, 0, 0};
    }

    // pages and scales of the next groups, a tile a lane; two sets, as loads run ahead of products
    int page = -1, page_next = -1;
    float ks = 0, vs = 0, ks_next = 0, vs_next = 0;
    auto look_up = [&](int gi, int &pg, float &k, float &v) {
        const int tile = tile_begin + gi * NT + lane;
        pg = tile < tile_end ? pool_page(c, seq, tile >> tile_shift) : -1;
        const int64_t slot = (int64_t)max(pg, 0) * c.heads + head;
        k = c.k_scales[slot];
        v = c.v_scales[slot];
    };
    uint4 kc[KU], vc[VU][2];
    auto load = [&](int gi) {                   // a step's codes, this wave's pieces
        if (gi % AHEAD == 0) look_up(gi, page_next, ks_next, vs_next);
        auto at = [&](const uint8_t *codes, int t, int j) {
            const int p = __builtin_amdgcn_readlane(page_next, (gi % AHEAD) * NT + t);
            const int64_t tile = (((int64_t)max(p, 0) * c.heads + head) << tile_shift) +
                                 ((tile_begin + gi * NT + t) & ((1 << tile_shift) - 1));
            return *(reinterpret_cast<const uint4 *>(codes + tile * (kTile * D) + 1024 * j) + lane);
        };
#pragma unroll
        for (int i = 0; i < KU; ++i) {
            const int piece = wave + kWaves * i;
            if (piece < NT * J) kc[i] = at(c.k, piece % NT, piece / NT);
        }
#pragma unroll
        for (int i = 0; i < VU; ++i) {
            const int piece = wave + kWaves * i;
            if (piece < NT / 2 * J) {
                vc[i][0] = at(c.v, piece % (NT / 2) * 2, piece / (NT / 2));
                vc[i][1] = at(c.v, piece % (NT / 2) * 2 + 1, piece / (NT / 2));
            }
        }
    };
    auto convert = [&](int gi) {                // what load() brought, into the buffer of step gi
        const int b = gi & 1;
#pragma unroll
        for (int i = 0; i < KU; ++i) {
            const int piece = wave + kWaves * i;
            if (piece >= NT * J) break;
            const int t = piece % NT, j = piece / NT;
            keys[b][t * 2 * J + 2 * j][lane] = __builtin_bit_cast(v4u, operand<FMT>(kc[i].x, kc[i].y));
            keys[b][t * 2 * J + 2 * j + 1][lane] = __builtin_bit_cast(v4u, operand<FMT>(kc[i].z, kc[i].w));
        }
#pragma unroll
        for (int i = 0; i < VU; ++i) {
            const int piece = wave + kWaves * i;
            if (piece >= NT / 2 * J) break;
            const int t = piece % (NT / 2) * 2, j = piece / (NT / 2);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // tokens that no row sees may hold anything: NaN codes must not meet the probability 0
                const int token = (tile_begin + gi * NT + t + h) * kTile;
                const bool there = __builtin_amdgcn_readlane(page_next, (gi % AHEAD) * NT + t + h) >= 0;
                if (!there || token < u.lo || token + kTile > u.up) {
                    uint32_t keep = 0;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (there && token + 4 * g + r >= u.lo && token + 4 * g + r < u.up) keep |= 0xFFu << (8 * r);
                    vc[i][h].x &= keep; vc[i][h].y &= keep; vc[i][h].z &= keep; vc[i][h].w &= keep;
                }
            }
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
                values[b][t / 2 * DT + 4 * j + d][lane] = w;
            }
        }
    };

    __syncthreads();                            // the buffers may still be read for the item before
    if (groups > 0) {
        load(0);
        convert(0);
        page = page_next; ks = ks_next; vs = vs_next;
    }
    if (groups > 1) load(1);
    __syncthreads();
    for (int gi = 0; gi < groups; ++gi) {
        const int b = gi & 1, tile0 = tile_begin + gi * NT;
        int mine[NT];
        float kf[NT], vf[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            mine[t] = __builtin_amdgcn_readlane(page, (gi % AHEAD) * NT + t);
            kf[t] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ks), (gi % AHEAD) * NT + t)) * a.scale;
            vf[t] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(vs), (gi % AHEAD) * NT + t));
        }
        if (gi + 1 < groups) {
            convert(gi + 1);
            if ((gi + 1) % AHEAD == 0) {
                page = page_next; ks = ks_next; vs = vs_next;
            }
        }
        if (gi + 2 < groups) load(gi + 2);
        const bool needed = tile0 * kTile < any.up && (tile0 + NT) * kTile > any.lo;
        if (needed) {
            bool edge = tile0 * kTile < all.lo || (tile0 + NT) * kTile > all.up;
#pragma unroll
            for (int t = 0; t < NT; ++t) edge |= mine[t] < 0;
            v4f x[RT][NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) x[rt][t] = v4f{0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < 2 * J; ++k) {
                    const v8bf kk = __builtin_bit_cast(v8bf, keys[b][t * 2 * J + k][lane]);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
                        x[rt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kk, q[rt][k], x[rt][t], 0, 0, 0);
                }
            }
            if (edge) {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int token = (tile0 + t) * kTile + 4 * g;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt)
                            x[rt][t][r] = mine[t] >= 0 && token + r >= seen[rt].lo && token + r < seen[rt].up
                                              ? x[rt][t][r] * kf[t]
                                              : -INFINITY;
                    kf[t] = 1.0f;
                    if (mine[t] < 0) vf[t] = 0.0f;       // the scale is another page's
                }
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                // x kf is the score: the scale of a tile is one for its maximum, and enters each power's argument
                float top = m[rt];
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    top = fmaxf(top, fmaxf(fmaxf(x[rt][t][0], x[rt][t][1]), fmaxf(x[rt][t][2], x[rt][t][3])) * kf[t]);
                top = row_max(top);
                const float from = top == -INFINITY ? 0.0f : top;
                if (__any(top > m[rt])) {
                    const float f = __builtin_amdgcn_exp2f(m[rt] - from);
                    l[rt] *= f;
#pragma unroll
                    for (int d = 0; d < DT; ++d) y[rt][d] *= f;
                    m[rt] = top;
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        x[rt][t][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[rt][t][r], kf[t], -from));
                        l[rt] += x[rt][t][r];
                    }
            }
#pragma unroll
            for (int t = 0; t < NT; t += 2) {
                if constexpr (F32) {
                    v8bf p[RT][TERMS];
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) terms<TERMS>(x[rt][t] * vf[t], x[rt][t + 1] * vf[t + 1], p[rt]);
#pragma unroll
                    for (int d = 0; d < DT; ++d) {
                        const v8bf v = __builtin_bit_cast(v8bf, values[b][t / 2 * DT + d][lane]);
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                            for (int n = 0; n < TERMS; ++n)
                                y[rt][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p[rt][n], y[rt][d], 0, 0, 0);
                    }
                } else {
                    // Base: a scale over 2^(base - 127) is between 2^-4 and 2^5, so a probability below
                    // fp16's normal numbers is off by 2^-21 of its value's magnitude at most.  A pair of tiles
                    // whose scales are further apart is multiplied a tile at a time.
                    const int e0 = vf[t] == 0.0f ? 0 : exponent(vf[t]), e1 = vf[t + 1] == 0.0f ? 0 : exponent(vf[t + 1]);
                    const int high = max(e0, e1), low = min(e0 ? e0 : high, e1 ? e1 : high);
                    const int rounds = high - low > 4 ? 2 : 1;
                    for (int round = 0; round < rounds; ++round) {
                        const int most = rounds == 1 ? high : round ? e1 : e0, least = rounds == 1 ? low : most;
                        if (most && (most > base + 4 || least < base - 4)) {
                            const int next = max(most, base - 80);      // sums of 2^30 tokens stay in fp32
                            const float f = __builtin_ldexpf(1.0f, max(base - next, -126));
#pragma unroll
                            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                                for (int d = 0; d < DT; ++d) y[rt][d] *= f;
                            base = next;
                        }
                        float f0 = __builtin_ldexpf(vf[t], 127 - base), f1 = __builtin_ldexpf(vf[t + 1], 127 - base);
                        if (rounds == 2) (round ? f0 : f1) = 0.0f;
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
                            const v8h v = __builtin_bit_cast(v8h, values[b][t / 2 * DT + d][lane]);
#pragma unroll
                            for (int rt = 0; rt < RT; ++rt)
                                y[rt][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, p[rt], y[rt][d], 0, 0, 0);
                        }
                    }
                }
            }
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
