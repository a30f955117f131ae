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
#include "qlin_device.h"

namespace qlin {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

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

__device__ __forceinline__ int adapter_of(const LoraLaunch &a, int id) {
    return (unsigned)id < (unsigned)a.adapters ? id : a.adapters;
}
__device__ __forceinline__ int rank_of(const LoraLaunch &a, int adapter) {
    if (adapter >= a.adapters) return 0;
    return a.ranks ? min(max(a.ranks[adapter], 0), a.max_rank) : a.max_rank;
}

constexpr int kShrinkWaves = 8, kShrinkWavesWide = 4;   // of a shrink workgroup, 16- and 64-row tiles

// One tile: `count` rows of one adapter (adapters: rows without one).
struct Tile {
    int adapter, count;
    int v0;   // row of v where the tile's first row is (-1: v has the call's row order)
};

// Rows up to which a workgroup finds its tile by ballots over the ids.
constexpr int kDirectRows = 64;

// Finds tile `ti` and its rows (member[0 .. 16 CT)); count 0: there is no
// such tile.  Ends with a barrier when the tile exists.
template <int CT, bool SORTED>
__device__ __forceinline__ Tile find_tile(const LoraLaunch &a, int ti, int *member) {
    Tile t = {0, 0, -1};
    const int tid = threadIdx.x, lane = tid & 63;
    if constexpr (SORTED) {
        if (ti >= a.tile_count[0]) return t;
        const int4 d = a.tiles[ti];
        t.adapter = d.x;
        t.v0 = d.y;
        t.count = d.z;
        if (tid < t.count) member[tid] = a.perm[d.y + tid];
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
    const int split = blockIdx.x, rank0 = blockIdx.z * 16 * RT;
    const Tile t = find_tile<CT, SORTED>(a, blockIdx.y, member);
    if (t.count == 0 || rank0 >= rank_of(a, t.adapter)) return;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int c16 = lane & 15, kg = lane >> 4;
    const uint16_t *xp[CT], *ap[RT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int i = c * 16 + c16;
        xp[c] = a.x + (int64_t)member[i < t.count ? i : 0] * a.ldx + kg * 8;
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int rank = min(rank0 + r * 16 + c16, a.max_rank - 1);
        ap[r] = a.A + ((int64_t)t.adapter * a.max_rank + rank) * a.K + kg * 8;
    }
    v4f acc[CT][RT] = {};
    const int s0 = (split * NW + w) * a.k_steps;
    const int s1 = min(s0 + a.k_steps, (a.K + 31) / 32);
#pragma unroll 4
    for (int s = s0; s < s1; ++s) {
        const int k = s * 32;
        const bool in = k + kg * 8 < a.K;   // K is a multiple of 16
        uint4 av[RT], xv[CT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
            av[r] = in ? *reinterpret_cast<const uint4 *>(ap[r] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int c = 0; c < CT; ++c)
            xv[c] = in ? *reinterpret_cast<const uint4 *>(xp[c] + k) : make_uint4(0, 0, 0, 0);
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

// y of one tile for n_chunk columns; each of the four waves has a quarter of
// them, 32 at a time.  D[column][row] from B rows and v.
//
// First the tile's v: the slices are added up, the adapter's scale is applied
// and the sum is written to the LDS as TERMS bf16 numbers that add up to it.
// Each takes 8 more bits of the mantissa, so that the second product loses
// nothing that its fp32 sums would keep (TERMS 3, fp32 y) or less than the
// bf16 rounding of y shows (TERMS 2).  Ranks past the adapter's are zero.
//
// RK: 32-rank steps (0: more than two, B read as it is needed).  The next
// columns' B rows and base are on their way while these are multiplied.  The
// columns of a wave's two tiles are dealt so that each lane ends with 16
// consecutive bytes of its row.
template <int CT, int RK, bool F32, bool SORTED>
__global__ __launch_bounds__(256) void expand_kernel(LoraLaunch a) {
    constexpr int TERMS = F32 ? 3 : 2, ROWS = 16 * CT;
    extern __shared__ __align__(16) uint16_t vs[];   // [TERMS][ROWS][stride]
    __shared__ int member[ROWS];
    const Tile t = find_tile<CT, SORTED>(a, blockIdx.y, member);
    if (t.count == 0) return;
    const int ranks = rank_of(a, t.adapter);
    if (ranks == 0 && a.base == a.y) return;   // these rows are already there
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int c16 = lane & 15, kg = lane >> 4;
    const int steps = RK > 0 ? RK : (ranks + 31) / 32, stride = steps * 32 + 8;
    const float scale = a.scales && t.adapter < a.adapters ? a.scales[t.adapter] : 1.0f;

    for (int i = tid; i < ROWS * steps * 8; i += 256) {   // four ranks of a row
        const int row = i / (steps * 8), rank = (i - row * steps * 8) * 4;
        v4f f = {0.0f, 0.0f, 0.0f, 0.0f};
        if (row < t.count && rank < ranks) {
            const float *p = a.v + (int64_t)(t.v0 >= 0 ? t.v0 + row : member[row]) * a.v_stride + rank;
            for (int s = 0; s < a.splits; ++s) f += *reinterpret_cast<const v4f *>(p + (int64_t)s * a.M * a.v_stride);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = rank + j < ranks ? f[j] * scale : 0.0f;
#pragma unroll
        for (int e = 0; e < TERMS; ++e) {
            const uint32_t lo = bf16_pair(f[0], f[1]), hi = bf16_pair(f[2], f[3]);
            *reinterpret_cast<uint2 *>(vs + ((int64_t)e * ROWS + row) * stride + rank) = make_uint2(lo, hi);
            f[0] -= bf16_lo(lo);
            f[1] -= bf16_hi(lo);
            f[2] -= bf16_lo(hi);
            f[3] -= bf16_hi(hi);
        }
    }
    __syncthreads();

    int64_t yrow[CT], brow[CT];
    bool in_tile[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        in_tile[c] = c * 16 + c16 < t.count;
        const int64_t m = member[in_tile[c] ? c * 16 + c16 : 0];
        yrow[c] = m * a.ldy;
        brow[c] = m * a.ldb;
    }
    const int quarter = a.n_chunk / 4;
    const int n_begin = blockIdx.x * a.n_chunk + w * quarter, n_end = min(a.N, n_begin + quarter);
    // D's row 4 kg + i of tile j is column col(j) + i, and the lane that loads
    // that row of B is c16 = 4 kg + i
    auto col = [&](int j, int g) { return F32 ? j * 16 + g * 4 : g * 8 + j * 4; };
    const uint16_t *bp[2];   // this lane's B row of tile j, at the wave's first column
#pragma unroll
    for (int j = 0; j < 2; ++j)
        bp[j] = a.B + ((int64_t)t.adapter * a.N + col(j, c16 >> 2) + (c16 & 3)) * a.max_rank + kg * 8;
    auto load_b = [&](int n, int q, uint4 (&b)[2]) {
        const int rank = q * 32 + kg * 8;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            b[j] = make_uint4(0, 0, 0, 0);
            if (rank < ranks && n + col(j, c16 >> 2) + (c16 & 3) < a.N)
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
    auto load_base = [&](int n, uint4 (&o)[CT][PARTS]) {
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int h = 0; h < PARTS; ++h) {
                const int at = n + col(h, kg);
                o[c][h] = make_uint4(0, 0, 0, 0);
                if (a.base && in_tile[c] && at < n_end) {
                    if constexpr (F32)
                        o[c][h] = *reinterpret_cast<const uint4 *>(static_cast<const float *>(a.base) + brow[c] + at);
                    else
                        o[c][h] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.base) + brow[c] + at);
                }
            }
    };
    constexpr int HELD = RK > 0 ? RK : 1;
    uint4 b_next[HELD][2], base_next[CT][PARTS];
    if constexpr (RK > 0)
#pragma unroll
        for (int q = 0; q < RK; ++q) load_b(n_begin, q, b_next[q]);
    load_base(n_begin, base_next);
    for (int n = n_begin; n < n_end; n += 32) {
        v4f acc[CT][2] = {};
        uint4 b_now[HELD][2], base_now[CT][PARTS];
        if constexpr (RK > 0) {
#pragma unroll
            for (int q = 0; q < RK; ++q)
#pragma unroll
                for (int j = 0; j < 2; ++j) b_now[q][j] = b_next[q][j];
        }
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int h = 0; h < PARTS; ++h) base_now[c][h] = base_next[c][h];
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
            clear_past(q, b);
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int e = TERMS - 1; e >= 0; --e) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(
                        vs + ((int64_t)e * ROWS + c * 16 + c16) * stride + q * 32 + kg * 8);
#pragma unroll
                    for (int j = 0; j < 2; ++j) acc[c][j] = mfma_bf16(b[j], v, acc[c][j]);
                }
            if constexpr (RK > 0)
                if (q + 1 == RK) break;
        }
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            if (!in_tile[c]) continue;
            if constexpr (F32) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int at = n + col(h, kg);
                    if (at < n_end)
                        *reinterpret_cast<v4f *>(static_cast<float *>(a.y) + yrow[c] + at) =
                            acc[c][h] + __builtin_bit_cast(v4f, base_now[c][h]);
                }
            } else {
                const int at = n + col(0, kg);
                const uint4 o = base_now[c][0];
                const v4f p = acc[c][0], q = acc[c][1];
                if (at < n_end)
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.y) + yrow[c] + at) =
                        make_uint4(bf16_pair(bf16_lo(o.x) + p[0], bf16_hi(o.x) + p[1]),
                                   bf16_pair(bf16_lo(o.y) + p[2], bf16_hi(o.y) + p[3]),
                                   bf16_pair(bf16_lo(o.z) + q[0], bf16_hi(o.z) + q[1]),
                                   bf16_pair(bf16_lo(o.w) + q[2], bf16_hi(o.w) + q[3]));
            }
        }
    }
}

// Sorts the rows by adapter (rows without one last) into perm, and cuts each
// adapter's rows into tiles.  One workgroup.  The order of an adapter's rows
// depends on which wave counts first; every row's result is the same in any
// place of any tile.
__global__ __launch_bounds__(1024) void group_kernel(LoraLaunch a, int tile_rows) {
    __shared__ uint32_t cnt[QLIN_MAX_ADAPTERS + 1];
    __shared__ uint32_t tot[2][16];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int n = a.adapters + 1;
    for (int i = tid; i < n; i += 1024) cnt[i] = 0;
    __syncthreads();
    // each row's place among its adapter's rows: within the wave by ballots
    // (one round for each adapter that the wave sees), across waves by one
    // atomic of the round's first lane
    for (int m0 = w * 64; m0 < a.M; m0 += 1024) {
        const int m = m0 + lane;
        const int id = m < a.M ? adapter_of(a, a.ids[m]) : -1;
        uint64_t todo = __ballot(m < a.M);
        int place = 0, lead = 0, count = 0;
        while (todo) {
            const int l = __ffsll((unsigned long long)todo) - 1;
            const uint64_t same = __ballot(id == __builtin_amdgcn_readlane(id, l));
            if (same >> lane & 1) {
                place = __popcll(same & ((1ull << lane) - 1));
                count = __popcll(same);
                lead = l;
            }
            todo &= ~same;
        }
        int before = 0;
        if (m < a.M && place == 0) before = (int)atomicAdd(&cnt[id], (uint32_t)count);
        before = __shfl(before, lead);
        if (m < a.M) a.place[m] = before + place;
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
    for (int m0 = w * 64; m0 < a.M; m0 += 1024) {
        const int m = m0 + lane;
        if (m < a.M) a.perm[cnt[adapter_of(a, a.ids[m])] + a.place[m]] = m;
    }
}

}  // namespace

// ---------------------------------------------------------------- planning

void lora_plan(int M, int N, int K, int adapters, int max_rank, LoraPlan *p) {
    p->sorted = M > kDirectRows;
    p->ct = M >= 1024 ? 4 : 1;
    const int tile_rows = 16 * p->ct;
    p->max_tiles = p->sorted ? (M + tile_rows - 1) / tile_rows + (adapters + 1 < M ? adapters + 1 : M) : M;
    p->rt = max_rank <= 16 ? 1 : max_rank <= 32 ? 2 : 4;
    p->rank_chunks = (max_rank + 16 * p->rt - 1) / (16 * p->rt);
    p->v_stride = (max_rank + 15) / 16 * 16;
    // K parts: one or two workgroups for each compute unit, at most four parts
    // (the expand kernel reads them all for each of its column runs), two
    // steps of 32 or more for each wave
    const int steps = (K + 31) / 32, waves = p->ct == 1 ? kShrinkWaves : kShrinkWavesWide;
    const int tiles = p->sorted ? (M + tile_rows - 1) / tile_rows : M;
    int splits = 2 * kComputeUnits / (tiles * p->rank_chunks);
    splits = splits > 4 ? 4 : splits < 1 ? 1 : splits;
    if (splits > steps / (2 * waves)) splits = steps / (2 * waves) > 0 ? steps / (2 * waves) : 1;
    p->k_steps = (steps + waves * splits - 1) / (waves * splits);
    p->splits = (steps + waves * p->k_steps - 1) / (waves * p->k_steps);
    // columns per expand workgroup: runs as long as leave four workgroups for
    // each compute unit
    int n_chunk = 256;
    while (n_chunk < 4096 && (int64_t)((N + 2 * n_chunk - 1) / (2 * n_chunk)) * tiles >= 4 * kComputeUnits) n_chunk *= 2;
    p->n_chunk = n_chunk;
    auto align = [](size_t v) { return (v + 255) & ~size_t(255); };
    size_t at = 0;
    p->v_at = at;
    at += align((size_t)p->splits * M * p->v_stride * 4);
    if (p->sorted) {
        p->tiles_at = at;
        at += align((size_t)p->max_tiles * 16);
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
    constexpr int NW = CT == 1 ? kShrinkWaves : kShrinkWavesWide;
    const dim3 grid(p.splits, p.max_tiles, p.rank_chunks), block(64 * NW);
    if (p.sorted) hipLaunchKernelGGL((shrink_kernel<CT, RT, NW, true>), grid, block, 0, s, a);
    else if constexpr (CT == 1) hipLaunchKernelGGL((shrink_kernel<CT, RT, NW, false>), grid, block, 0, s, a);
}

template <int CT, int RK, bool F32>
static void launch_expand(const LoraPlan &p, const LoraLaunch &a, hipStream_t s) {
    const dim3 grid((a.N + p.n_chunk - 1) / p.n_chunk, p.max_tiles), block(256);
    const int steps = RK > 0 ? RK : (a.max_rank + 31) / 32;
    const size_t lds = (size_t)(F32 ? 3 : 2) * 16 * CT * (steps * 32 + 8) * 2;
    if (p.sorted) hipLaunchKernelGGL((expand_kernel<CT, RK, F32, true>), grid, block, lds, s, a);
    else if constexpr (CT == 1) hipLaunchKernelGGL((expand_kernel<CT, RK, F32, false>), grid, block, lds, s, a);
}

template <int CT>
static hipError_t launch_products(const LoraPlan &p, bool f32, const LoraLaunch &a, hipStream_t s) {
    if (p.rt == 1) launch_shrink<CT, 1>(p, a, s);
    else if (p.rt == 2) launch_shrink<CT, 2>(p, a, s);
    else launch_shrink<CT, 4>(p, a, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int steps = (a.max_rank + 31) / 32;
    if (steps == 1) f32 ? launch_expand<CT, 1, true>(p, a, s) : launch_expand<CT, 1, false>(p, a, s);
    else if (steps == 2) f32 ? launch_expand<CT, 2, true>(p, a, s) : launch_expand<CT, 2, false>(p, a, s);
    else f32 ? launch_expand<CT, 0, true>(p, a, s) : launch_expand<CT, 0, false>(p, a, s);
    return hipGetLastError();
}

hipError_t launch_lora(const LoraPlan &p, bool f32, const LoraLaunch &a, hipStream_t s) {
    if (p.sorted) {
        hipLaunchKernelGGL(group_kernel, dim3(1), dim3(1024), 0, s, a, 16 * p.ct);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return p.ct == 1 ? launch_products<1>(p, f32, a, s) : launch_products<4>(p, f32, a, s);
}

}  // namespace qlin
