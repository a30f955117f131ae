// qlin_lora.hip -- low-rank adapters of many requests beside a shared
// projection: y[m] = base[m] + s_a B_a (A_a x[m]) with a = ids[m].
//
// Two products with a tall and a wide thin matrix, on the bf16 matrix cores.
// Rows of one adapter share its weights, so both kernels work on tiles of
// rows of one adapter:
//   shrink  v = A_a x over a part of K, kept in fp32 in the workspace, one
//           slice for each part;
//   expand  adds the slices up and y = base + s B_a v for a run of columns.
// Up to 64 rows, a workgroup finds its tile from the ids with one ballot;
// past that, group_kernel sorts the rows by adapter first.
#include <algorithm>

#include "qlin_device.h"

namespace qlin {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v4f mfma_bf16(uint4 a, uint4 b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0,
                                                   0);
}

// two fp32 -> two bf16, nearest even, NaN kept
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    v2bf p;
    p[0] = (__bf16)lo;
    p[1] = (__bf16)hi;
    return __builtin_bit_cast(uint32_t, p);
}

// A fragment of the matrix cores has lane 16 c + r hold chunk c (16 bytes, 8
// numbers of the common axis) of row r.  Loaded like that, neighbouring lanes
// lie in different rows and each is an access of its own: 64 clocks of a
// compute unit's address unit for a wave's KiB.  So lane 4 r + c loads it,
// four lanes for 64 consecutive bytes (16 clocks), and the lanes change
// places.
__device__ __forceinline__ uint4 to_fragment(uint4 v, int from) {
    return make_uint4((uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v.x),
                      (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v.y),
                      (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v.z),
                      (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v.w));
}
// the lane whose chunk becomes this lane's, in bytes
__device__ __forceinline__ int fragment_source(int lane) { return ((lane & 15) * 4 + (lane >> 4)) * 4; }

__device__ __forceinline__ int adapter_of(const LoraLaunch &a, int id) {
    return (unsigned)id < (unsigned)a.adapters ? id : a.adapters;
}
__device__ __forceinline__ int rank_of(const LoraLaunch &a, int adapter) {
    if (adapter >= a.adapters) return 0;
    return a.ranks ? min(max(a.ranks[adapter], 0), a.max_rank) : a.max_rank;
}

constexpr int kShrinkWaves = 8;   // of a shrink workgroup

constexpr int kWideRows = 64;   // rows of a wide tile

// One tile: `count` rows of one adapter (adapters: rows without one).
struct Tile {
    int adapter, count;
    int v0;   // row of v where the tile's first row is (-1: v has the call's row order)
};

// Rows up to which a workgroup finds its tile by ballots over the ids.
constexpr int kDirectRows = 64;

// Finds part `sub` (16 CT rows) of tile `ti` and its rows (member[0 .. 16 CT));
// count 0: there is no such part.  Ends with a barrier when there is.
template <int CT, bool SORTED>
__device__ __forceinline__ Tile find_tile(const LoraLaunch &a, int ti, int sub, int *member) {
    Tile t = {0, 0, -1};
    const int tid = threadIdx.x, lane = tid & 63;
    if constexpr (SORTED) {
        if (ti >= a.tile_count[0]) return t;
        const int4 d = a.tiles[ti];
        const int first = sub * 16 * CT;
        if (first >= d.z) return t;
        t.adapter = d.x;
        t.v0 = d.y + first;
        t.count = min(d.z - first, 16 * CT);
        if (tid < t.count) member[tid] = a.perm[t.v0 + tid];
    } else {
        // a tile starts at every 16th row of its adapter's rows, and is known
        // by that row's number
        const int lead = adapter_of(a, a.ids[ti]);
        uint64_t same[kDirectRows / 64];
        int before = 0, all = 0;
#pragma unroll
        for (int q = 0; q < kDirectRows / 64; ++q) {
            const int m = q * 64 + lane;
            same[q] = __ballot(m < a.M && adapter_of(a, a.ids[m < a.M ? m : 0]) == lead);
            all += __popcll(same[q]);
            before += __popcll(ti >= q * 64 + 64 ? same[q] : ti > q * 64 ? same[q] & ((1ull << (ti - q * 64)) - 1) : 0);
        }
        if (before & 15) return t;
        t.adapter = lead;
        t.count = min(16, all - before);
        if (tid < 64) {
            int at = -before;
#pragma unroll
            for (int q = 0; q < kDirectRows / 64; ++q) {
                const int place = at + __popcll(same[q] & ((1ull << lane) - 1));
                if ((same[q] >> lane & 1) && place >= 0 && place < 16) member[place] = q * 64 + lane;
                at += __popcll(same[q]);
            }
        }
    }
    __syncthreads();
    return t;
}

// v (a part of K) for one tile and 16 RT ranks: D[rank][row] from A rows and
// x rows, both read along K.  The NW waves split the part's K steps and add
// up through the LDS, 16 rows at a time.
template <int CT, int RT, int NW, bool SORTED>
__global__ __launch_bounds__(64 * NW) void shrink_kernel(LoraLaunch a) {
    __shared__ int member[16 * CT];
    __shared__ v4f part[NW][RT][64];
    // grid x: K part, then row tile's part (2^20 rows are more than grid y holds)
    const int split = blockIdx.x % a.splits, part_of = blockIdx.x / a.splits, rank0 = blockIdx.y * 16 * RT;
    const Tile t = find_tile<CT, SORTED>(a, part_of / a.sub_tiles, part_of % a.sub_tiles, member);
    // (the first ranks are computed whether the adapter has them or not: their
    // loads do not wait for its rank)
    if (t.count == 0 || t.adapter >= a.adapters || (rank0 > 0 && rank0 >= rank_of(a, t.adapter))) return;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int c16 = lane & 15, kg = lane >> 4;
    // this lane's part of the loads: row lane / 4, chunk lane % 4
    const int from = fragment_source(lane), lrow = lane >> 2, lk = (lane & 3) * 8;
    const uint16_t *xp[CT], *ap[RT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int i = c * 16 + lrow;
        xp[c] = a.x + (int64_t)member[i < t.count ? i : 0] * a.ldx + lk;
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int rank = min(rank0 + r * 16 + lrow, a.max_rank - 1);
        ap[r] = a.A + ((int64_t)t.adapter * a.max_rank + rank) * a.K + lk;
    }
    v4f acc[CT][RT] = {};
    const int s0 = (split * NW + w) * a.k_steps;
    const int s1 = min(s0 + a.k_steps, (a.K + 31) / 32);
#pragma unroll 4
    for (int s = s0; s < s1; ++s) {
        const int k = s * 32;
        const bool in = k + lk < a.K;   // K is a multiple of 16
        uint4 av[RT], xv[CT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
            av[r] = in ? *reinterpret_cast<const uint4 *>(ap[r] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int c = 0; c < CT; ++c)
            xv[c] = in ? *reinterpret_cast<const uint4 *>(xp[c] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < RT; ++r) av[r] = to_fragment(av[r], from);
#pragma unroll
        for (int c = 0; c < CT; ++c) xv[c] = to_fragment(xv[c], from);
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int r = 0; r < RT; ++r) acc[c][r] = mfma_bf16(av[r], xv[c], acc[c][r]);
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        if (c * 16 >= t.count) break;
        if (c > 0) __syncthreads();
#pragma unroll
        for (int r = 0; r < RT; ++r) part[w][r][lane] = acc[c][r];
        __syncthreads();
        const int i = c * 16 + c16;
        for (int r = w; r < RT; r += NW) {
            v4f s = part[0][r][lane];
#pragma unroll
            for (int q = 1; q < NW; ++q) s += part[q][r][lane];
            if (i >= t.count || rank0 + r * 16 >= a.v_stride) continue;
            const int64_t row = t.v0 >= 0 ? t.v0 + i : member[i];
            *reinterpret_cast<v4f *>(a.v + ((int64_t)split * a.M + row) * a.v_stride + rank0 + r * 16 + kg * 4) = s;
        }
    }
}

// What bf16 number `hi` leaves of f; nothing where it is infinite (inf - inf
// would turn an infinite product into NaN).
__device__ __forceinline__ float left_of(float f, float hi) {
    const float r = f - hi;
    return __builtin_fabsf(r) < INFINITY ? r : 0.0f;
}

// A number between the products is this many bf16 numbers that add up to it:
// each takes 8 more bits of the mantissa, so three keep the 24 bits of fp32.
// Two would be 1 to 2 % faster for ranks up to 64 (3 to 6 % for 256; 4096 rows
// of rank 64: 70.4 us against 71.0) but lose what B's products leave where
// they cancel across the ranks.
constexpr int kTerms = 3;

__device__ __forceinline__ void split4(v4f f, uint2 (&out)[kTerms]) {
#pragma unroll
    for (int e = 0; e < kTerms; ++e) {
        out[e] = make_uint2(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]));
        f[0] = left_of(f[0], bf16_lo(out[e].x));
        f[1] = left_of(f[1], bf16_hi(out[e].x));
        f[2] = left_of(f[2], bf16_lo(out[e].y));
        f[3] = left_of(f[3], bf16_hi(out[e].y));
    }
}

// Eight bf16 columns: base + what the products give, each rounded once.
__device__ __forceinline__ uint4 add_pairs(uint4 b, float f0, float f1, float f2, float f3, float f4, float f5, float f6,
                                           float f7) {
    return make_uint4(bf16_pair(bf16_lo(b.x) + f0, bf16_hi(b.x) + f1), bf16_pair(bf16_lo(b.y) + f2, bf16_hi(b.y) + f3),
                      bf16_pair(bf16_lo(b.z) + f4, bf16_hi(b.z) + f5), bf16_pair(bf16_lo(b.w) + f6, bf16_hi(b.w) + f7));
}

// A tile's v into the LDS (vs[kTerms][ROWS][32 steps + 8]) by 256 threads: the
// slices are added up, the adapter's scale is applied and the sum is kept as
// kTerms bf16 numbers.  Ranks past the adapter's are zero.
template <int ROWS>
__device__ __forceinline__ void fill_v(const LoraLaunch &a, const Tile &t, const int *member, int ranks, int steps,
                                       uint16_t *vs) {
    const int tid = threadIdx.x, stride = steps * 32 + 8;
    const float scale = a.scales && t.adapter < a.adapters ? a.scales[t.adapter] : 1.0f;
    for (int row = tid >> 4; row < ROWS; row += 16)   // 16 threads a row, four ranks each
        for (int rank = (tid & 15) * 4; rank < steps * 32; rank += 64) {
            v4f f = {0.0f, 0.0f, 0.0f, 0.0f};
            if (row < t.count && rank < ranks) {
                const float *p = a.v + (int64_t)(t.v0 >= 0 ? t.v0 + row : member[row]) * a.v_stride + rank;
                for (int s = 0; s < a.splits; ++s) f += *reinterpret_cast<const v4f *>(p + (int64_t)s * a.M * a.v_stride);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = rank + j < ranks ? f[j] * scale : 0.0f;
            uint2 o[kTerms];
            split4(f, o);
#pragma unroll
            for (int e = 0; e < kTerms; ++e) *reinterpret_cast<uint2 *>(vs + (e * ROWS + row) * stride + rank) = o[e];
        }
}

// y of one tile of up to 16 rows for n_chunk columns; each of the four waves
// has a quarter of them, 32 at a time.  D[column][row] from B rows and v.
//
// RK: 32-rank steps (0: more than two, B read as it is needed).  The next
// columns' B rows and base are on their way while these are multiplied.  The
// columns of a wave's two tiles are dealt so that each lane ends with 16
// consecutive bytes of its row.
template <int RK, bool F32, bool SORTED>
__global__ __launch_bounds__(256, 4) void expand_kernel(LoraLaunch a) {
    extern __shared__ __align__(16) uint16_t vs[];   // [kTerms][16][stride]
    __shared__ int member[16];
    const Tile t = find_tile<1, SORTED>(a, blockIdx.y, 0, member);
    if (t.count == 0) return;
    const int ranks = rank_of(a, t.adapter);
    if (ranks == 0 && a.base == a.y) return;   // these rows are already there
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int c16 = lane & 15, kg = lane >> 4;
    const int steps = RK > 0 ? RK : (ranks + 31) / 32, stride = steps * 32 + 8;

    const bool in_tile = c16 < t.count;
    const int64_t m = member[in_tile ? c16 : 0], yrow = m * a.ldy, brow = m * a.ldb;
    const int quarter = a.n_chunk / 4;
    const int n_begin = blockIdx.x * a.n_chunk + w * quarter, n_end = min(a.N, n_begin + quarter);
    // D's row 4 kg + i of tile j is column col(j, kg) + i, and so is row 4 kg + i
    // of its fragment of B
    auto col = [&](int j, int g) { return F32 ? j * 16 + g * 4 : g * 8 + j * 4; };
    const int from = fragment_source(lane), lrow = lane >> 2, lrank = (lane & 3) * 8;
    const uint16_t *bp[2];   // the B row of tile j that this lane loads from, at the call's first column
#pragma unroll
    for (int j = 0; j < 2; ++j)
        bp[j] = a.B + ((int64_t)t.adapter * a.N + col(j, lrow >> 2) + (lrow & 3)) * a.max_rank + lrank;
    // single tokens load what max_rank covers, without waiting for the rank;
    // sorted rows, where B's bytes are what takes the time, only the adapter's
    const int loaded = SORTED ? ranks : t.adapter < a.adapters ? a.max_rank : 0;
    auto load_b = [&](int n, int q, uint4 (&b)[2]) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            b[j] = make_uint4(0, 0, 0, 0);
            if (q * 32 + lrank < loaded && n + col(j, lrow >> 2) + (lrow & 3) < a.N)
                b[j] = *reinterpret_cast<const uint4 *>(bp[j] + (int64_t)n * a.max_rank + q * 32);
        }
    };
    // ranks past the adapter's: whatever B holds there is cleared
    auto clear_past = [&](int q, uint4 (&b)[2]) {
        if ((q + 1) * 32 <= ranks) return;
        const int rank = q * 32 + kg * 8;
        uint32_t keep[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            keep[i] = (rank + 2 * i < ranks ? 0xFFFFu : 0u) | (rank + 2 * i + 1 < ranks ? 0xFFFF0000u : 0u);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            b[j] = make_uint4(b[j].x & keep[0], b[j].y & keep[1], b[j].z & keep[2], b[j].w & keep[3]);
    };
    constexpr int PARTS = F32 ? 2 : 1;   // 16-byte pieces of a lane's columns
    auto load_base = [&](int n, uint4 (&o)[PARTS]) {
#pragma unroll
        for (int h = 0; h < PARTS; ++h) {
            const int at = n + col(h, kg);
            o[h] = make_uint4(0, 0, 0, 0);
            if (a.base && in_tile && at < n_end) {
                if constexpr (F32)
                    o[h] = *reinterpret_cast<const uint4 *>(static_cast<const float *>(a.base) + brow + at);
                else
                    o[h] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.base) + brow + at);
            }
        }
    };
    // many rows' y leaves with the non-temporal policy (see expand_wide_kernel;
    // 2048 rows, 4096 columns of fp32, K 12288: 38 us against 44)
    auto put = [](void *to, v4u v) {
        if constexpr (SORTED) __builtin_nontemporal_store(v, static_cast<v4u *>(to));
        else *static_cast<v4u *>(to) = v;
    };
    constexpr int HELD = RK > 0 ? RK : 1;
    uint4 b_next[HELD][2], base_next[PARTS];
    if constexpr (RK > 0)
#pragma unroll
        for (int q = 0; q < RK; ++q) load_b(n_begin, q, b_next[q]);
    load_base(n_begin, base_next);

    fill_v<16>(a, t, member, ranks, steps, vs);
    __syncthreads();

    for (int n = n_begin; n < n_end; n += 32) {
        v4f acc[2] = {};
        uint4 b_now[HELD][2], base_now[PARTS];
        if constexpr (RK > 0) {
#pragma unroll
            for (int q = 0; q < RK; ++q)
#pragma unroll
                for (int j = 0; j < 2; ++j) b_now[q][j] = b_next[q][j];
        }
#pragma unroll
        for (int h = 0; h < PARTS; ++h) base_now[h] = base_next[h];
        if (n + 32 < n_end) {
            if constexpr (RK > 0)
#pragma unroll
                for (int q = 0; q < RK; ++q) load_b(n + 32, q, b_next[q]);
            load_base(n + 32, base_next);
        }
        for (int q = 0; q < steps; ++q) {
            uint4 b[2];
            if constexpr (RK == 0) {
                load_b(n, q, b);
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j) b[j] = b_now[RK == 1 ? 0 : q][j];
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) b[j] = to_fragment(b[j], from);
            clear_past(q, b);
#pragma unroll
            for (int e = kTerms - 1; e >= 0; --e) {
                const uint4 v = *reinterpret_cast<const uint4 *>(vs + (e * 16 + c16) * stride + q * 32 + kg * 8);
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[j] = mfma_bf16(b[j], v, acc[j]);
            }
            if constexpr (RK > 0)
                if (q + 1 == RK) break;
        }
        if (!in_tile) continue;
        if constexpr (F32) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = n + col(h, kg);
                if (at < n_end)
                    put(static_cast<float *>(a.y) + yrow + at,
                        __builtin_bit_cast(v4u, acc[h] + __builtin_bit_cast(v4f, base_now[h])));
            }
        } else {
            const int at = n + col(0, kg);
            if (at < n_end)
                put(static_cast<uint16_t *>(a.y) + yrow + at,
                    __builtin_bit_cast(v4u, add_pairs(base_now[0], acc[0][0], acc[0][1], acc[0][2], acc[0][3], acc[1][0],
                                                      acc[1][1], acc[1][2], acc[1][3])));
        }
    }
}

// y of one tile of up to 64 rows (16 a wave) for n_chunk columns, COLS at a
// time.  D[row][column] from v and B rows.
//
// What bounds it is the way to memory, and that is a matter of how neighbouring
// lanes lie.  A fragment of the matrix cores has them in different rows: read
// or written like that, every lane is an access of its own, 16 bytes a clock
// for a compute unit.  So B goes through the LDS, loaded as it lies in memory
// a stage ahead, once for 64 rows; and a lane has NJ consecutive columns (tile
// j has the columns NJ c + j), so that 16 lanes load and store 256 consecutive
// bytes of a row of y, with the non-temporal policy (the next call's shrink
// then does not wait for y's lines to leave the caches: 27 -> 21 us).  4096
// rows, 10240 columns, rank 64: 45 us (with two terms of v 44, against 62 with
// B read by each wave and half lines of y at a time, 55 with 128 bytes of a
// row).
//   PASS  8-rank chunks of B in a stage: 4 (max_rank <= 32) or 8
//   ONE   a stage holds all ranks (max_rank <= 8 PASS): v stays in registers
template <int PASS, bool ONE, bool F32>
__global__ __launch_bounds__(256) void expand_wide_kernel(LoraLaunch a) {
    constexpr int ROWS = kWideRows, NJ = F32 ? 4 : 8, COLS = 16 * NJ;
    constexpr int LOADS = COLS * PASS / 256;              // 16-byte loads of a thread for a stage
    __shared__ uint4 bs[COLS * (PASS + 1)];               // [tile j, lane's column][chunk], rows one chunk apart
    extern __shared__ __align__(16) uint16_t vs[];        // [kTerms][ROWS][stride]
    __shared__ int member[ROWS];
    const Tile t = find_tile<ROWS / 16, true>(a, blockIdx.y, 0, member);
    if (t.count == 0) return;
    const int ranks = rank_of(a, t.adapter);
    if (ranks == 0 && a.base == a.y) return;   // these rows are already there
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int c16 = lane & 15, kg = lane >> 4;
    const int steps = (a.max_rank + 31) / 32, stride = steps * 32 + 8;
    const int n_begin = blockIdx.x * a.n_chunk, n_end = min(a.N, n_begin + a.n_chunk);
    const int held = min(a.max_rank / 8, PASS);           // chunks of a B row in a stage
    const int passes = ONE ? (ranks > 0 ? 1 : 0) : (ranks + PASS * 8 - 1) / (PASS * 8);

    // chunk p of a stage is column p / held (by its reciprocal: exact for
    // p < 2^13), place p % held; it goes to the LDS row of its tile and lane
    const uint32_t recip = 65536u / held + 1;
    int to[LOADS], from[LOADS], place[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int p = i * 256 + tid, col = (int)(p * recip >> 16);
        place[i] = p - col * held;
        to[i] = ((col % NJ) * 16 + col / NJ) * (PASS + 1) + place[i];
        from[i] = col * a.max_rank + place[i] * 8;
        if (col >= COLS) place[i] = 1 << 20;   // past the stage
    }
    const uint16_t *const b_rows = a.B + (int64_t)t.adapter * a.N * a.max_rank;
    uint4 next[LOADS];
    auto load_b = [&](int n, int pass) {
        const uint16_t *p = b_rows + (int64_t)n * a.max_rank + pass * PASS * 8;
        if (held == PASS && n + COLS <= n_end && (pass + 1) * PASS * 8 <= ranks) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) next[i] = *reinterpret_cast<const uint4 *>(p + from[i]);
            return;
        }
        const int end = (n_end - n) * a.max_rank - pass * PASS * 8;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            next[i] = make_uint4(0, 0, 0, 0);
            if ((pass * PASS + place[i]) * 8 < ranks && from[i] < end) next[i] = *reinterpret_cast<const uint4 *>(p + from[i]);
        }
    };
    auto put_b = [&]() {
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            if (place[i] < held) bs[to[i]] = next[i];
    };
    load_b(n_begin, 0);

    fill_v<ROWS>(a, t, member, ranks, steps, vs);
    put_b();
    __syncthreads();

    const int row0 = w * 16;
    const bool idle = row0 >= t.count;
    const v4u *const base0 = static_cast<const v4u *>(a.base);
    v4u *const y0 = static_cast<v4u *>(a.y);
    constexpr int PER = F32 ? 4 : 8;   // columns of 16 bytes
    int64_t base_at[4], y_at[4];
    bool live[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = row0 + kg * 4 + i;
        live[i] = r < t.count;
        const int64_t m = member[live[i] ? r : 0];
        base_at[i] = (m * a.ldb + n_begin) / PER + c16;
        y_at[i] = (m * a.ldy + n_begin) / PER + c16;
    }
    uint4 vf[PASS / 4][kTerms];
    auto load_v = [&](int pass) {
#pragma unroll
        for (int q = 0; q < PASS / 4; ++q)
#pragma unroll
            for (int e = 0; e < kTerms; ++e)
                vf[q][e] = pass * PASS * 8 + q * 32 < ranks
                               ? *reinterpret_cast<const uint4 *>(vs + (e * ROWS + row0 + c16) * stride + pass * PASS * 8 +
                                                                  q * 32 + kg * 8)
                               : make_uint4(0, 0, 0, 0);
    };
    if constexpr (ONE) load_v(0);
    for (int n = n_begin; n < n_end; n += COLS) {
        const bool in = n + c16 * PER < n_end;   // n_end is a multiple of 16
        v4u base[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            base[i] = v4u{0, 0, 0, 0};
            if (a.base && in && live[i]) base[i] = __builtin_nontemporal_load(base0 + base_at[i]);
            base_at[i] += COLS / PER;
        }
        v4f acc[NJ] = {};
        for (int pass = 0; pass < passes; ++pass) {
            const bool more = pass + 1 < passes || n + COLS < n_end;
            if (pass + 1 < passes) load_b(n, pass + 1);
            else if (n + COLS < n_end) load_b(n + COLS, 0);
            if constexpr (!ONE) load_v(pass);
#pragma unroll
            for (int q = 0; q < PASS / 4; ++q) {
                const int rank0 = pass * PASS * 8 + q * 32, rank = rank0 + kg * 8;
                if (rank0 >= ranks || idle) break;
                uint4 bq[NJ];
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    bq[j] = bs[(j * 16 + c16) * (PASS + 1) + q * 4 + kg];
                if (rank0 + 32 > ranks) {   // as expand_kernel's clear_past
                    uint32_t keep[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        keep[i] = (rank + 2 * i < ranks ? 0xFFFFu : 0u) | (rank + 2 * i + 1 < ranks ? 0xFFFF0000u : 0u);
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        bq[j] = make_uint4(bq[j].x & keep[0], bq[j].y & keep[1], bq[j].z & keep[2], bq[j].w & keep[3]);
                }
#pragma unroll
                for (int e = kTerms - 1; e >= 0; --e)
#pragma unroll
                    for (int j = 0; j < NJ; ++j) acc[j] = mfma_bf16(vf[q][e], bq[j], acc[j]);
            }
            if (more) {
                __syncthreads();
                put_b();
                __syncthreads();
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v4u o;
            if constexpr (F32) {
                o = __builtin_bit_cast(v4u, v4f{acc[0][i], acc[1][i], acc[2][i], acc[3][i]} + __builtin_bit_cast(v4f, base[i]));
            } else {
                o = __builtin_bit_cast(v4u, add_pairs(__builtin_bit_cast(uint4, base[i]), acc[0][i], acc[1][i], acc[2][i],
                                                      acc[3][i], acc[4][i], acc[5][i], acc[6][i], acc[7][i]));
            }
            if (in && live[i]) __builtin_nontemporal_store(o, y0 + y_at[i]);
            y_at[i] += COLS / PER;
        }
    }
}

// A lane's partner in a DPP step.
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ float moved(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROW_MASK, 0xF, false));
}
// The wave's sum, in lane 63 (steps as in wave_max).
__device__ __forceinline__ float wave_add(float v) {
    v += moved<0xB1>(v);
    v += moved<0x4E>(v);
    v += moved<0x141>(v);
    v += moved<0x140>(v);
    v += moved<0x142, 0xA>(v);
    return v + moved<0x143, 0xC>(v);
}
// sum + p . q of eight bf16 each
__device__ __forceinline__ float dot8(uint4 p, uint4 q, float sum) {
    const uint32_t u[4] = {p.x, p.y, p.z, p.w}, v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sum = __builtin_fmaf(bf16_lo(u[i]), bf16_lo(v[i]), sum);
        sum = __builtin_fmaf(bf16_hi(u[i]), bf16_hi(v[i]), sum);
    }
    return sum;
}

// Both products for one row in one launch, on the vector ALUs: for a few
// single tokens the second launch costs more than reading the row's A again in
// every workgroup.  v stays in fp32.
//
// Wave w takes the ranks w, w + 8, ...: the lanes lie along K, so A comes in
// 1 KiB of consecutive bytes a load.  Then P lanes take a column, 8 ranks
// each.  B and base are on their way meanwhile.
template <int P, bool F32>
__global__ __launch_bounds__(512) void few_rows_kernel(LoraLaunch a) {
    __shared__ float v[8 * P];
    constexpr int PER = 512 / P;   // columns of a workgroup
    const int m = blockIdx.y, tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int adapter = adapter_of(a, a.ids[m]), ranks = rank_of(a, adapter);
    const int n = blockIdx.x * PER + tid / P, rank0 = tid % P * 8;
    const int64_t at = (int64_t)m * a.ldy + n;
    const bool first = tid % P == 0 && n < a.N;
    // A and B are loaded as far as max_rank, without waiting for the rank
    const int loaded = adapter < a.adapters ? a.max_rank : 0;
    uint4 b = make_uint4(0, 0, 0, 0);
    if (n < a.N && rank0 < loaded)
        b = *reinterpret_cast<const uint4 *>(a.B + ((int64_t)adapter * a.N + n) * a.max_rank + rank0);
    float base = 0.0f;
    if (first && a.base) {
        const int64_t from = (int64_t)m * a.ldb + n;
        if constexpr (F32) base = static_cast<const float *>(a.base)[from];
        else base = __uint_as_float((uint32_t) static_cast<const uint16_t *>(a.base)[from] << 16);
    }
    const float scale = a.scales && adapter < a.adapters ? a.scales[adapter] : 1.0f;
    const uint16_t *x = a.x + (int64_t)m * a.ldx;
    for (int r = w; r < 8 * P; r += 8) {
        float sum = 0.0f;
        if (r < loaded) {
            const uint16_t *row = a.A + ((int64_t)adapter * a.max_rank + r) * a.K;
#pragma unroll 4
            for (int k = lane * 8; k < a.K; k += 512) {
                const uint4 p = *reinterpret_cast<const uint4 *>(row + k), q = *reinterpret_cast<const uint4 *>(x + k);
                sum = dot8(p, q, sum);
            }
        }
        sum = wave_add(sum);
        if (lane == 63) v[r] = sum * scale;
    }
    __syncthreads();
    float y = 0.0f;
    const uint32_t q[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {   // ranks past the adapter's: whatever B holds there is not used
        const float f = i & 1 ? bf16_hi(q[i / 2]) : bf16_lo(q[i / 2]);
        y = rank0 + i < ranks ? __builtin_fmaf(f, v[rank0 + i], y) : y;
    }
    if constexpr (P > 1) y = y + moved<0xB1>(y);
    if constexpr (P > 2) y = y + moved<0x4E>(y);
    if constexpr (P > 4) y = y + moved<0x141>(y);
    if (!first || (ranks == 0 && a.base == a.y)) return;   // a row without ranks is already there, every bit of it
    if constexpr (F32) static_cast<float *>(a.y)[at] = base + y;
    else static_cast<uint16_t *>(a.y)[at] = (uint16_t)bf16_pair(base + y, 0.0f);
}

// Sorts the rows by adapter (rows without one last) into perm, and cuts each
// adapter's rows into tiles.  One workgroup.  The order of an adapter's rows
// depends on which wave counts first; every row's result is the same in any
// place of any tile.
constexpr int kHeldRows = 4, kRounds = 4;

__global__ __launch_bounds__(1024) void group_kernel(LoraLaunch a, int tile_rows) {
    __shared__ uint32_t cnt[QLIN_MAX_ADAPTERS + 1];
    __shared__ uint32_t tot[2][16];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int n = a.adapters + 1;
    for (int i = tid; i < n; i += 1024) cnt[i] = 0;
    __syncthreads();
    // each row's place among its adapter's rows: within the wave by ballots, a
    // round for each of the first adapters that the wave sees (long runs have
    // few), with one atomic of the round's first lane; the other rows by an
    // atomic each.  A thread's first rows stay in registers.
    int ids[kHeldRows], places[kHeldRows];
    auto count = [&](int id, bool live) {
        uint64_t todo = __ballot(live);
        int place = 0, lead = lane, rows = 1;
        for (int round = 0; round < kRounds && todo; ++round) {
            const int l = __ffsll((unsigned long long)todo) - 1;
            const uint64_t same = __ballot(id == __builtin_amdgcn_readlane(id, l));
            if (same >> lane & 1) {
                place = __popcll(same & ((1ull << lane) - 1));
                rows = __popcll(same);
                lead = l;
            }
            todo &= ~same;
        }
        int before = 0;
        if (live && place == 0) before = (int)atomicAdd(&cnt[id], (uint32_t)rows);
        return __shfl(before, lead) + place;
    };
#pragma unroll
    for (int q = 0; q < kHeldRows; ++q) {
        const int m = q * 1024 + tid;
        ids[q] = m < a.M ? adapter_of(a, a.ids[m]) : -1;
    }
#pragma unroll
    for (int q = 0; q < kHeldRows; ++q)
        if (q * 1024 + w * 64 < a.M) places[q] = count(ids[q], ids[q] >= 0);
    for (int m0 = kHeldRows * 1024 + w * 64; m0 < a.M; m0 += 1024) {
        const int m = m0 + lane;
        const int place = count(m < a.M ? adapter_of(a, a.ids[m]) : -1, m < a.M);
        if (m < a.M) a.place[m] = place;
    }
    __syncthreads();
    // exclusive sums of the rows and of the tiles, a run of adapters per thread
    const int per = (n + 1023) / 1024;
    uint32_t rows = 0, tiles = 0;
    for (int i = tid * per; i < min(n, tid * per + per); ++i) {
        rows += cnt[i];
        tiles += (cnt[i] + tile_rows - 1) / tile_rows;
    }
    uint32_t r = rows, q = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t ur = __shfl_up(r, d), uq = __shfl_up(q, d);
        if (lane >= d) {
            r += ur;
            q += uq;
        }
    }
    if (lane == 63) {
        tot[0][w] = r;
        tot[1][w] = q;
    }
    __syncthreads();
    r -= rows;
    q -= tiles;
    for (int i = 0; i < w; ++i) {
        r += tot[0][i];
        q += tot[1][i];
    }
    for (int i = tid * per; i < min(n, tid * per + per); ++i) {
        const uint32_t c = cnt[i];
        cnt[i] = r;
        for (uint32_t d = 0; d < c; d += tile_rows)
            a.tiles[q++] = make_int4(i, (int)(r + d), (int)min(c - d, (uint32_t)tile_rows), 0);
        r += c;
    }
    if (tid == 1023) a.tile_count[0] = (int)q;   // the last run ends after every tile
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kHeldRows; ++q)
        if (ids[q] >= 0) a.perm[cnt[ids[q]] + places[q]] = q * 1024 + tid;
    for (int m = kHeldRows * 1024 + tid; m < a.M; m += 1024) a.perm[cnt[adapter_of(a, a.ids[m])] + a.place[m]] = m;
}

}  // namespace

// ---------------------------------------------------------------- planning

// Whether tiles are wide (64 rows, each B row read once for them instead of
// every 16 rows, and base and y in longer pieces).  Wide tiles pay where B is
// read often (rows x rank) or where base and y come from HBM; before that the
// narrow ones, of which there are four times as many, fill the compute units
// better.  Narrow / wide (time), with new x and base each call, six adapters
// in runs of 251 rows and 64 with single rows:
//   rank 8   10240 x 5120: 2000 rows (82 MB of base and y) 0.92, 0.97; 3000 1.30, 1.07
//            4096 x 4096: 3000 rows (49 MB) 0.92, 0.86; 4000 1.07, 1.07; 2048 x 2048: 6000 0.95, 0.87
//   rank 32  4096 x 4096: 3000 rows 0.95, 0.96; 4000 1.15, 1.22
//   rank 64  2048 x 6144: 2000 rows 0.82, 0.98; 3000 1.12, 1.23; 10240 x 5120: 1536 rows 0.99, 1.17; 2000 1.19, 1.27
//   rank 256 4096 x 4096: 2000 rows 1.08, 0.89; 3000 0.89, 1.29
//   fp32     10240 x 5120: rank 8, 1100 rows (90 MB) 1.01, 0.87; 1536 1.16, 1.01; rank 32, 1100 rows 0.90, 1.05
// With x and base still in the caches narrow tiles stay ahead for longer, for
// ranks up to 16 by 5 to 15 %.
static bool wide_tiles(int M, int N, int max_rank, bool f32) {
    if (M < 1280) return false;
    return (int64_t)M * N * (f32 ? 8 : 4) >= 80000000 || (int64_t)M * std::min(max_rank, 48) >= 120000;
}

// One launch for both products: where a row's A is small, so that reading it
// in every workgroup costs less than a second launch.  In elements of A: a
// row's, all rows', and what all workgroups read together.  Inside these
// bounds (times: in a replayed graph, an adapter for each row) 3.9 us against
// 7.0 (rank 16, 4096 x 2048, 1 row), 6.1 against 8.4 (rank 16, 10240 x 5120, 4
// rows), 8.5 against 8.6 (rank 64, 2048 x 2048, 2); outside 9.3 against 8.5
// (rank 32, 10240 x 5120, 1 row), 12.5 against 8.7 (the same, 4 rows), 9.2
// against 8.8 (rank 64, 2048 x 2048, 8).  Small ranks would gain from a few
// rows more: 5.6 against 8.0 (rank 16, 4096 x 4096, 16).
static bool few_rows(int M, int N, int K, int max_rank) {
    if (M > 16 || max_rank > 64) return false;
    const int lanes = max_rank <= 8 ? 1 : max_rank <= 16 ? 2 : max_rank <= 32 ? 4 : 8;   // of a column
    const int64_t one = (int64_t)K * max_rank, groups = (int64_t)M * ((N + 512 / lanes - 1) / (512 / lanes));
    return one <= 1 << 17 && M * one <= 1 << 19 && groups * one <= 1 << 24;
}

void lora_plan(int M, int N, int K, int adapters, int max_rank, bool f32, LoraPlan *p) {
    p->few = few_rows(M, N, K, max_rank);
    p->sorted = M > kDirectRows;
    p->wide = wide_tiles(M, N, max_rank, f32);
    const int tile_rows = p->wide ? kWideRows : 16;
    p->max_tiles = p->sorted ? (M + tile_rows - 1) / tile_rows + std::min(adapters + 1, M) : M;
    p->rt = max_rank <= 16 ? 1 : max_rank <= 32 ? 2 : 4;
    p->rank_chunks = (max_rank + 16 * p->rt - 1) / (16 * p->rt);
    p->v_stride = (max_rank + 15) / 16 * 16;
    // K parts: two workgroups for each compute unit, two steps of 32 or more
    // for each wave.  At most four parts, two for wide tiles: every expand
    // workgroup reads them all (4096 rows of rank 64: four take 2 % longer than
    // two).  Up to 32 rows eight, as many as let a wave's loads leave at once
    // (rank 64, K 12288: 16 rows 14.3 us against 17.3 with four; 64 rows 33.8
    // against 30.3).
    p->shrink_ct = p->wide && p->rt > 1 ? 2 : 1;
    p->sub_tiles = tile_rows / (16 * p->shrink_ct);
    const int steps = (K + 31) / 32, waves = kShrinkWaves;
    const int groups = std::min(adapters, M);
    // about how many tiles there are: full ones, or one for each adapter
    const int tiles = std::max((M + tile_rows - 1) / tile_rows, groups);
    const int shrink_tiles = std::max((M + 16 * p->shrink_ct - 1) / (16 * p->shrink_ct), groups);
    int splits = 2 * kComputeUnits / (shrink_tiles * p->rank_chunks);
    const int few_cap = std::min(std::max(steps / (4 * waves), 4), 8), most = std::max(steps / (2 * waves), 1);
    const int cap = p->wide ? 2 : M > 32 ? 4 : few_cap;
    splits = std::min({std::max(splits, 1), cap, most});
    p->k_steps = (steps + waves * splits - 1) / (waves * splits);
    p->splits = (steps + waves * p->k_steps - 1) / (waves * p->k_steps);
    // columns per expand workgroup: four stages of the wide kernel, or runs
    // as long as leave eight workgroups for each compute unit
    int n_chunk = 256;
    if (p->wide) {
        n_chunk = f32 ? 256 : 512;
    } else {
        while (n_chunk < 4096 && (int64_t)((N + 2 * n_chunk - 1) / (2 * n_chunk)) * tiles >= 8 * kComputeUnits) n_chunk *= 2;
    }
    p->n_chunk = n_chunk;
    auto align = [](size_t v) { return (v + 255) & ~size_t(255); };
    // The workspace holds what any call of at most M rows takes, so that one
    // sized for the most rows serves fewer: rows of v in all slices, which are
    // M in one, up to few_cap slices of 32 rows, or up to four slices of which
    // two workgroups for each compute unit, of at most 32 rows, write; and
    // tiles of 16 rows.
    const int64_t v_rows = std::max({(int64_t)M, (int64_t)std::min(M, 32) * std::min(few_cap, most),
                                     std::min((int64_t)M * std::min(4, most), (int64_t)2 * kComputeUnits * 32)});
    size_t at = 0;
    p->v_at = at;
    at += align((size_t)v_rows * p->v_stride * 4);
    if (p->sorted) {
        p->tiles_at = at;
        at += align((size_t)((M + 15) / 16 + std::min(adapters + 1, M)) * 16);
        p->count_at = at;
        at += 256;
        p->perm_at = at;
        at += align((size_t)M * 4);
        p->place_at = at;
        at += align((size_t)M * 4);
    }
    p->ws_bytes = at;
}

template <int CT, int RT>
static void launch_shrink(const LoraPlan &p, const LoraLaunch &a, hipStream_t s) {
    constexpr int NW = kShrinkWaves;
    const dim3 grid(p.splits * p.max_tiles * p.sub_tiles, p.rank_chunks), block(64 * NW);
    if (p.sorted) hipLaunchKernelGGL((shrink_kernel<CT, RT, NW, true>), grid, block, 0, s, a);
    else if constexpr (CT == 1) hipLaunchKernelGGL((shrink_kernel<CT, RT, NW, false>), grid, block, 0, s, a);
}

template <int RK, bool F32>
static void launch_expand(const LoraPlan &p, const LoraLaunch &a, hipStream_t s) {
    const dim3 grid((a.N + p.n_chunk - 1) / p.n_chunk, p.max_tiles), block(256);
    const int steps = RK > 0 ? RK : (a.max_rank + 31) / 32;
    const size_t lds = (size_t)kTerms * 16 * (steps * 32 + 8) * 2;
    if (p.sorted) hipLaunchKernelGGL((expand_kernel<RK, F32, true>), grid, block, lds, s, a);
    else hipLaunchKernelGGL((expand_kernel<RK, F32, false>), grid, block, lds, s, a);
}

template <int PASS, bool ONE, bool F32>
static void launch_expand_wide(const LoraPlan &p, const LoraLaunch &a, hipStream_t s) {
    const dim3 grid((a.N + p.n_chunk - 1) / p.n_chunk, p.max_tiles), block(256);
    const size_t lds = (size_t)kTerms * kWideRows * ((a.max_rank + 31) / 32 * 32 + 8) * 2;
    hipLaunchKernelGGL((expand_wide_kernel<PASS, ONE, F32>), grid, block, lds, s, a);
}

template <bool F32>
static void launch_expand_any(const LoraPlan &p, const LoraLaunch &a, hipStream_t s) {
    if (p.wide) {
        if (a.max_rank <= 32) launch_expand_wide<4, true, F32>(p, a, s);
        else if (a.max_rank <= 64) launch_expand_wide<8, true, F32>(p, a, s);
        else launch_expand_wide<8, false, F32>(p, a, s);
    } else {
        if (a.max_rank <= 32) launch_expand<1, F32>(p, a, s);
        else if (a.max_rank <= 64) launch_expand<2, F32>(p, a, s);
        else launch_expand<0, F32>(p, a, s);
    }
}

template <int P>
static void launch_few_rows(bool f32, const LoraLaunch &a, hipStream_t s) {
    const dim3 grid((a.N + 512 / P - 1) / (512 / P), a.M), block(512);
    if (f32) hipLaunchKernelGGL((few_rows_kernel<P, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((few_rows_kernel<P, false>), grid, block, 0, s, a);
}

hipError_t launch_lora(const LoraPlan &p, bool f32, const LoraLaunch &a, hipStream_t s) {
    hipError_t e = hipSuccess;
    if (p.few) {
        if (a.max_rank <= 8) launch_few_rows<1>(f32, a, s);
        else if (a.max_rank <= 16) launch_few_rows<2>(f32, a, s);
        else if (a.max_rank <= 32) launch_few_rows<4>(f32, a, s);
        else launch_few_rows<8>(f32, a, s);
        return hipGetLastError();
    }
    if (p.sorted) {
        hipLaunchKernelGGL(group_kernel, dim3(1), dim3(1024), 0, s, a, p.wide ? kWideRows : 16);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (p.rt == 1) launch_shrink<1, 1>(p, a, s);
    else if (p.rt == 2) p.shrink_ct == 1 ? launch_shrink<1, 2>(p, a, s) : launch_shrink<2, 2>(p, a, s);
    else p.shrink_ct == 1 ? launch_shrink<1, 4>(p, a, s) : launch_shrink<2, 4>(p, a, s);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (f32) launch_expand_any<true>(p, a, s);
    else launch_expand_any<false>(p, a, s);
    return hipGetLastError();
}

}  // namespace qlin
