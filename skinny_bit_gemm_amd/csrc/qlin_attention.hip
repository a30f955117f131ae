// qlin_attention.hip -- attention over the paged 8-bit cache.
//
//   y = sum_j p_j v_j / sum_j p_j,  p_j = 2^(x_j - max x),  x_j = log2(e) scale q . k_j
//
// One pass over a sequence's tokens with a running maximum and sum.  Both
// products run transposed on the bf16 matrix cores, with the codes as their left
// operands: S^T = K Q^T, then Y^T = V^T P^T.  A lane then has one query row in
// the scores, in the running maximum and sum, and in Y^T alike, and the scores
// of two tiles of 16 tokens are the second product's operand as they stand: no
// value changes lanes but the maximum.  The cache's tiles are stored in the order
// of these operands, so every load of a wave is 1 KiB of consecutive codes.
// e4m3 and int8 codes are bf16 numbers, so products with them are exact; the
// scales of a page multiply the scores and the probabilities.  Probabilities
// enter the second product as two bf16 terms (16 bits of mantissa; three, 24
// bits, where y is fp32): one term alone costs as much again as the rounding of y.
#include <algorithm>

#include "qlin_sequences.h"

namespace qlin {

namespace {

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kTile = 16;
constexpr int kWaves = 4;
constexpr int kMaxParts = 256;

// four codes of a word as bf16 (exact)
template <int FMT>
__device__ __forceinline__ uint2 bf16_codes(uint32_t w) {
    if constexpr (FMT == FMT_I8) {
        const uint32_t f0 = __float_as_uint((float)(int8_t)w), f1 = __float_as_uint((float)(int8_t)(w >> 8));
        const uint32_t f2 = __float_as_uint((float)(int8_t)(w >> 16)), f3 = __float_as_uint((float)(int8_t)(w >> 24));
        return make_uint2(__builtin_amdgcn_perm(f1, f0, 0x07060302u), __builtin_amdgcn_perm(f3, f2, 0x07060302u));
    }
    return make_uint2(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)));
}

// eight codes as a matrix operand
template <int FMT>
__device__ __forceinline__ v8bf operand(uint32_t lo, uint32_t hi) {
    const uint2 a = bf16_codes<FMT>(lo), b = bf16_codes<FMT>(hi);
    return __builtin_bit_cast(v8bf, v4u{a.x, a.y, b.x, b.y});
}

// over the four lanes l, l ^ 16, l ^ 32, l ^ 48 of a query row
__device__ __forceinline__ float row_max(float v) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float row_sum(float v) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// The rows of a workgroup (unit) and the tokens that they see.
struct Unit {
    int seq, row0, rows;       // first row (token x group + head of the group), rows that are there
    Sequence q;
    int lo, up;                // tokens that any row sees
    int all_lo, all_up;        // tokens that every row sees
    int tile0, tiles;          // tiles of 16 tokens of [lo, up)
};

struct Seen {
    int lo, up;
};
__device__ __forceinline__ Seen seen_by(const AttentionLaunch &a, const Sequence &q, int token) {
    const int p = q.start + token;
    Seen s;
    s.up = a.causal ? min(q.length, p + 1) : q.length;
    s.lo = a.window > 0 ? (int)max((int64_t)0, (int64_t)p + 1 - a.window) : 0;
    return s;
}

template <int ROWS>
__device__ __forceinline__ bool unit_of(const AttentionLaunch &a, Unit *u) {
    int within;
    u->seq = unit_sequence(
        a.c, blockIdx.x,
        [&](const Sequence &q) { return (int)min(((int64_t)q.n * a.group + ROWS - 1) / ROWS, (int64_t)1 << 24); },
        &within);
    if (u->seq < 0) return false;
    u->q = sequence_at(a.c, u->seq);
    u->row0 = within * ROWS;
    u->rows = min(ROWS, u->q.n * a.group - u->row0);
    const Seen first = seen_by(a, u->q, u->row0 / a.group), last = seen_by(a, u->q, (u->row0 + u->rows - 1) / a.group);
    u->lo = first.lo;
    u->up = last.up;
    u->all_lo = last.lo;
    u->all_up = first.up;
    u->tile0 = u->lo / kTile;
    u->tiles = u->up > u->lo ? (u->up + kTile - 1) / kTile - u->tile0 : 0;
    return true;
}

// parts that a unit's tokens are in (one at least)
__device__ __forceinline__ int parts_of(const AttentionLaunch &a, const Unit &u) {
    const int per = a.chunk / kTile;
    return max(1, min(a.parts, (u.tiles + per - 1) / per));
}

template <bool F32>
__device__ __forceinline__ void store_y4(void *y, int64_t at, v4f v) {
    if constexpr (F32) {
        *reinterpret_cast<v4f *>(static_cast<float *>(y) + at) = v;
    } else {
        const v4bf b = {(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
        *reinterpret_cast<v4bf *>(static_cast<uint16_t *>(y) + at) = b;
    }
}

// element of y (or of q) where a unit's row and this head's channels begin
__device__ __forceinline__ int64_t row_at(const AttentionLaunch &a, const Unit &u, int row, int64_t ld, int head, int D) {
    const int r = u.row0 + row, token = r / a.group;
    return (int64_t)(u.q.first + token) * ld + (int64_t)(head * a.group + r - token * a.group) * D;
}

// RT: tiles of 16 query rows; all waves have the same rows and take groups of NT
// tiles of tokens in turn, so a code is read and converted once for all rows.
template <int D, int FMT, int TERMS, int RT>
__global__ __launch_bounds__(64 * kWaves) void attention_kernel(AttentionLaunch a) {
    constexpr int ROWS = 16 * RT, J = D / 64, DT = D / 16, NT = D <= 128 ? 4 : 2;
    constexpr int AHEAD = 64 / NT;              // groups whose pages a wave looks up at once
    constexpr bool F32 = TERMS == 3;
    __shared__ float merge[kWaves][16][D + 4];
    __shared__ float2 merge_ml[kWaves][16];
    const CacheArgs &c = a.c;
    const int head = blockIdx.y, part = blockIdx.z;
    Unit u;
    if (!unit_of<ROWS>(a, &u)) return;
    const int parts = parts_of(a, u);
    if (part >= parts) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, col = lane & 15;
    const int tile_begin = u.tile0 + part * (a.chunk / kTile);
    const int tile_end = part == a.parts - 1 ? u.tile0 + u.tiles : min(u.tile0 + u.tiles, tile_begin + a.chunk / kTile);

    v8bf q[RT][2 * J];
    Seen seen[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int row = min(rt * 16 + col, u.rows - 1);
        const uint16_t *from = a.q + row_at(a, u, row, a.ldq, head, D);
#pragma unroll
        for (int k = 0; k < 2 * J; ++k)
            q[rt][k] = *reinterpret_cast<const v8bf *>(from + 64 * (k >> 1) + 16 * g + 8 * (k & 1));
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
    const int groups = (tile_end - tile_begin + NT - 1) / NT;
    int page = -1;
    float ks = 0.0f, vs = 0.0f;
    for (int gi = wave, k = 0; gi < groups; gi += kWaves, ++k) {
        if (k % AHEAD == 0) {                   // pages and scales of the next groups, a tile a lane
            const int tile = tile_begin + (gi + kWaves * (lane / NT)) * NT + lane % NT;
            page = tile < tile_end ? pool_page(c, u.seq, tile >> tile_shift) : -1;
            const int64_t slot = (int64_t)max(page, 0) * c.heads + head;
            ks = c.k_scales[slot];
            vs = c.v_scales[slot];
        }
        const int lane0 = (k % AHEAD) * NT, tile0 = tile_begin + gi * NT;
        uint4 kc[NT][J], vc[NT][J];
        float kf[NT], vf[NT];
        bool edge = tile0 * kTile < u.all_lo || (tile0 + NT) * kTile > u.all_up;
        int there[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            there[t] = __builtin_amdgcn_readlane(page, lane0 + t);
            edge |= there[t] < 0;
            kf[t] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ks), lane0 + t)) * a.scale;
            vf[t] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(vs), lane0 + t));
            const int64_t tile = (((int64_t)max(there[t], 0) * c.heads + head) << tile_shift) +
                                 ((tile0 + t) & ((1 << tile_shift) - 1));
            const uint4 *kp = reinterpret_cast<const uint4 *>(c.k + tile * (kTile * D)) + lane;
            const uint4 *vp = reinterpret_cast<const uint4 *>(c.v + tile * (kTile * D)) + lane;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                kc[t][j] = kp[64 * j];
                vc[t][j] = vp[64 * j];
            }
        }
        // scores: row token 4 g + r of tile t, column the lane's query row
        v4f x[RT][NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) x[rt][t] = v4f{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const v8bf k0 = operand<FMT>(kc[t][j].x, kc[t][j].y), k1 = operand<FMT>(kc[t][j].z, kc[t][j].w);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    x[rt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, q[rt][2 * j], x[rt][t], 0, 0, 0);
                    x[rt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, q[rt][2 * j + 1], x[rt][t], 0, 0, 0);
                }
            }
        }
        if (edge) {
            // tokens that no row sees may hold anything: NaN codes must not meet the probability 0
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int token = (tile0 + t) * kTile + 4 * g;
                uint32_t keep = 0;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool any = there[t] >= 0 && token + r >= u.lo && token + r < u.up;
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
                if (there[t] < 0) vf[t] = 0.0f;      // the scale is another page's
            }
        } else {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) x[rt][t] *= kf[t];
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            float top = m[rt];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) top = fmaxf(top, x[rt][t][r]);
            top = row_max(top);
            const float from = top == -INFINITY ? 0.0f : top;    // nothing seen yet: all p are 0
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
                    x[rt][t][r] = __builtin_amdgcn_exp2f(x[rt][t][r] - from);
                    l[rt] += x[rt][t][r];
                    x[rt][t][r] *= vf[t];
                }
        }
        // second product, 32 tokens at a time
#pragma unroll
        for (int t = 0; t < NT; t += 2) {
            v8bf p[RT][TERMS];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float rest = x[rt][t + (i >> 2)][i & 3];
#pragma unroll
                    for (int n = 0; n < TERMS; ++n) {
                        p[rt][n][i] = (__bf16)rest;
                        rest -= (float)p[rt][n][i];
                    }
                }
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const uint4 &v0 = vc[t][d >> 2], &v1 = vc[t + 1][d >> 2];
                const uint32_t w0 = (d & 3) == 0 ? v0.x : (d & 3) == 1 ? v0.y : (d & 3) == 2 ? v0.z : v0.w;
                const uint32_t w1 = (d & 3) == 0 ? v1.x : (d & 3) == 1 ? v1.y : (d & 3) == 2 ? v1.z : v1.w;
                const v8bf v = operand<FMT>(w0, w1);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int n = 0; n < TERMS; ++n)
                        y[rt][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p[rt][n], y[rt][d], 0, 0, 0);
            }
        }
    }

    // the waves' sums together, 16 rows at a time
    const int64_t slot = ((int64_t)part * a.units + blockIdx.x) * c.heads + head;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        if (rt) __syncthreads();
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
            if (parts == 1) store_y4<F32>(a.y, to + d, v * by);
            else *reinterpret_cast<v4f *>(a.part_o + (slot * ROWS + row) * D + d) = v;
        }
        if (parts > 1 && (threadIdx.x & 15) == 0) a.part_ml[slot * ROWS + row] = make_float2(top, total);
    }
}

// The parts of a unit's row together: a workgroup each.
template <int D, bool F32, int ROWS>
__global__ __launch_bounds__(256) void join_kernel(AttentionLaunch a) {
    constexpr int LANES = D / 4, SETS = 256 / LANES;
    __shared__ float factor[kMaxParts];
    __shared__ v4f sums[SETS][LANES];
    __shared__ float red[2][4];
    Unit u;
    if (!unit_of<ROWS>(a, &u)) return;
    const int head = blockIdx.y, row = blockIdx.z, tid = threadIdx.x;
    const int parts = parts_of(a, u);
    if (row >= u.rows || parts == 1) return;
    const int64_t step = (int64_t)a.units * a.c.heads * ROWS;
    const int64_t at = ((int64_t)blockIdx.x * a.c.heads + head) * ROWS + row;
    float2 ml = make_float2(-INFINITY, 0.0f);
    if (tid < parts) ml = a.part_ml[tid * step + at];
    const float top_w = wave_max(ml.x);
    if ((tid & 63) == 0) red[0][tid >> 6] = top_w;
    __syncthreads();
    const float top = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    const float f = ml.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml.x - top);
    factor[tid] = f;
    float sum = f * ml.y;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
    if ((tid & 63) == 0) red[1][tid >> 6] = sum;
    __syncthreads();
    const float total = red[1][0] + red[1][1] + red[1][2] + red[1][3];
    const int set = tid / LANES, d = 4 * (tid % LANES);
    if (set < SETS) {
        v4f v = {0, 0, 0, 0};
        for (int p = set; p < parts; p += SETS)
            v += *reinterpret_cast<const v4f *>(a.part_o + (p * step + at) * D + d) * factor[p];
        sums[set][tid % LANES] = v;
    }
    __syncthreads();
    if (tid < LANES) {
        v4f v = sums[0][tid];
        for (int s = 1; s < SETS; ++s) v += sums[s][tid];
        store_y4<F32>(a.y, row_at(a, u, row, a.ldy, head, D) + 4 * tid, v * (total > 0.0f ? 1.0f / total : 0.0f));
    }
}

template <int D, int FMT, int TERMS, int RT>
void launch_rows(const AttentionPlan &p, const AttentionLaunch &a, hipStream_t s) {
    hipLaunchKernelGGL((attention_kernel<D, FMT, TERMS, RT>), dim3(a.units, a.c.heads, a.parts), dim3(64 * kWaves), 0, s, a);
    if (a.parts > 1)
        hipLaunchKernelGGL((join_kernel<D, TERMS == 3, 16 * RT>), dim3(a.units, a.c.heads, 16 * RT), dim3(256), 0, s, a);
}

template <int D, int FMT>
void launch_width(bool f32, const AttentionPlan &p, const AttentionLaunch &a, hipStream_t s) {
    if (p.rows == 16) f32 ? launch_rows<D, FMT, 3, 1>(p, a, s) : launch_rows<D, FMT, 2, 1>(p, a, s);
    else f32 ? launch_rows<D, FMT, 3, 2>(p, a, s) : launch_rows<D, FMT, 2, 2>(p, a, s);
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

constexpr int kSlots = 2048;       // (unit, head, part) workgroups that a split call aims at, at most
constexpr int kMinChunk = 512;     // tokens of a part, at least

int64_t most_parts(int max_context) {
    return std::min<int64_t>(kMaxParts, std::max<int64_t>(1, (max_context + kMinChunk - 1) / kMinChunk));
}

}  // namespace

AttentionPlan attention_plan(int sequences, int tokens, int max_context, int kv_heads, int group, int head_dim) {
    AttentionPlan p = {};
    if (sequences == 0 || tokens == 0) return p;
    p.rows = (int64_t)tokens * group <= 16 * (int64_t)sequences ? 16 : 32;
    p.units = row_tiles(sequences, tokens, group, p.rows);
    const int64_t most = most_parts(max_context);
    p.parts = (int)std::max<int64_t>(1, std::min(most, kSlots / (p.units * kv_heads)));
    p.chunk = (int)(((int64_t)max_context + p.parts - 1) / p.parts + 255) / 256 * 256;   // whole groups of each wave
    // the workspace of the calls with as many or fewer sequences, tokens, and context
    const int64_t slots = std::min<int64_t>(kSlots, row_tiles(sequences, tokens, group, 16) * kv_heads * most);
    if (most > 1) {
        p.ml_at = (size_t)slots * 32 * head_dim * sizeof(float);
        p.ws_bytes = p.ml_at + (size_t)slots * 32 * sizeof(float2);
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
