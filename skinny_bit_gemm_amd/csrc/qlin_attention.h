// qlin_attention.h -- what the attention kernels share: codes as operands of the
// matrix cores, probabilities as theirs, and the rows and tokens of a unit of work.
//
//   y = sum_j p_j v_j / sum_j p_j,  p_j = 2^(x_j - max x),  x_j = log2(e) scale q . k_j
//
// One pass over a sequence's tokens with a running maximum and sum.  Both
// products run transposed on the matrix cores, with the codes as their left
// operands: S^T = K Q^T, then Y^T = V^T P^T.  A lane then has one query row in
// the scores, in the running maximum and sum, and in Y^T alike, and the scores
// of two tiles of 16 tokens are the second product's operand as they stand: no
// value changes lanes but the maximum.  The cache's tiles are stored in the order
// of these operands, so every load of a wave is 1 KiB of consecutive codes.
// e4m3 and int8 codes are bf16 numbers, so products with them are exact; the
// scales of a page multiply the scores and the probabilities.
#pragma once

#include "qlin_sequences.h"

namespace qlin {

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kTile = 16;
constexpr int kWaves = 4;

// four codes of a word as bf16 (exact)
template <int FMT>
__device__ __forceinline__ uint2 bf16_codes(uint32_t w) {
    if constexpr (FMT == FMT_I8) {
        asm("" : "+v"(w));      // one register until here: its bytes are not taken apart when it is loaded
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

typedef float v2f __attribute__((ext_vector_type(2)));

// eight probabilities as TERMS operands, whose sum has 8 bits of mantissa from each
template <int TERMS>
__device__ __forceinline__ void terms(v4f a, v4f b, v8bf (&p)[TERMS]) {
    v2f rest[4] = {{a[0], a[1]}, {a[2], a[3]}, {b[0], b[1]}, {b[2], b[3]}};
#pragma unroll
    for (int n = 0; n < TERMS; ++n) {
        v4u w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(rest[i], v2bf));     // nearest even
            if (n + 1 < TERMS) {
                rest[i][0] -= bf16_lo(w[i]);
                rest[i][1] -= bf16_hi(w[i]);
            }
        }
        p[n] = __builtin_bit_cast(v8bf, w);
    }
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

// A unit of work: a tile of a sequence's query rows (token x group + head of the
// group), and the tokens that they see.
struct Unit {
    int seq, row0, rows;       // first row, rows that are there
    Sequence q;
    int lo, up;                // tokens that any row sees
    int all_lo, all_up;        // tokens that every row sees
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

__device__ __forceinline__ Unit unit_at(const AttentionLaunch &a, int seq, const Sequence &q, int tile, int tile_rows) {
    Unit u;
    u.seq = seq;
    u.q = q;
    u.row0 = tile * tile_rows;
    u.rows = min(tile_rows, q.n * a.group - u.row0);
    const Seen first = seen_by(a, q, u.row0 / a.group), last = seen_by(a, q, (u.row0 + u.rows - 1) / a.group);
    u.lo = first.lo;
    u.up = last.up;
    u.all_lo = last.lo;
    u.all_up = first.up;
    return u;
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

// a row's operand of the first product: channels 64 (k / 2) + 16 g + 8 (k % 2) ..
__device__ __forceinline__ v8bf query(const AttentionLaunch &a, const uint16_t *from, int k, int g) {
    const v4u w = *reinterpret_cast<const v4u *>(from + 64 * (k >> 1) + 16 * g + 8 * (k & 1));
    return __builtin_bit_cast(v8bf, w ^ a.flip);
}

// element of y (or of q) where a unit's row and this head's channels begin
__device__ __forceinline__ int64_t row_at(const AttentionLaunch &a, const Unit &u, int row, int64_t ld, int head, int D) {
    const int r = u.row0 + row, token = r / a.group;
    return (int64_t)(u.q.first + token) * ld + (int64_t)(head * a.group + r - token * a.group) * D;
}

// a value that all lanes have, in scalar registers
__device__ __forceinline__ int64_t uniform(int64_t v) {
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)v) |
                     (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32);
}

__device__ __forceinline__ int64_t readlane(int64_t v, int lane) {
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)v, lane) |
                     (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32);
}

__device__ __forceinline__ Sequence uniform(const Sequence &q) {
    Sequence r;
    r.first = __builtin_amdgcn_readfirstlane(q.first);
    r.n = __builtin_amdgcn_readfirstlane(q.n);
    r.start = __builtin_amdgcn_readfirstlane(q.start);
    r.length = __builtin_amdgcn_readfirstlane(q.length);
    return r;
}

}  // namespace qlin
