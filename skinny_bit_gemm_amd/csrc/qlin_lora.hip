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

// One tile: `count` rows of one adapter (adapters: rows without one).
struct Tile {
    int adapter, count;
    int v0;   // row of v where the tile's first row is (-1: v has the call's row order)
};

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
        // the tile's first row is row ti, and every 16th of its adapter's
        // rows is one
        const int mine = lane < a.M ? adapter_of(a, a.ids[lane]) : -1;
        const int lead = __builtin_amdgcn_readlane(mine, ti);
        const uint64_t same = __ballot(mine == lead);
        const int before = __popcll(same & ((1ull << ti) - 1));
        if (before & 15) return t;
        const int at = __popcll(same & ((1ull << lane) - 1)) - before;
        t.adapter = lead;
        t.count = min(16, __popcll(same) - before);
        if (tid < 64 && mine == lead && at >= 0 && at < 16) member[at] = lane;
    }
    __syncthreads();
    return t;
}

// v (a part of K) for one tile and 16 RT ranks: D[rank][row] from A rows and
// x rows, both read along K.  The four waves split the part's K steps and add
// up through the LDS.
template <int CT, int RT, bool SORTED>
__global__ __launch_bounds__(256) void shrink_kernel(LoraLaunch a) {
    __shared__ int member[16 * CT];
    __shared__ v4f part[3][CT * RT][64];
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
    const int s0 = (split * 4 + w) * a.k_steps;
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
    if (w > 0) {
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int r = 0; r < RT; ++r) part[w - 1][c * RT + r][lane] = acc[c][r];
    }
    __syncthreads();
    if (w > 0) return;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int i = c * 16 + c16;
        if (i >= t.count) continue;
        const int64_t row = t.v0 >= 0 ? t.v0 + i : member[i];
        float *v = a.v + ((int64_t)split * a.M + row) * a.v_stride + rank0 + kg * 4;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            v4f s = acc[c][r];
            for (int q = 0; q < 3; ++q) s += part[q][c * RT + r][lane];
            if (rank0 + r * 16 < a.v_stride) *reinterpret_cast<v4f *>(v + r * 16) = s;
        }
    }
}

// The sum of v's slices for one row and the ranks kg * 8 + 0 .. 7 of a step
// of 32, times the adapter's scale, as TERMS bf16 numbers that add up to it:
// each takes 8 more bits of the mantissa, so that the second product loses
// nothing that its fp32 sums would keep (TERMS 3) or less than the bf16
// rounding of y would show (TERMS 2).  Ranks past the adapter's are zero.
template <int TERMS>
__device__ __forceinline__ void load_v(const LoraLaunch &a, int64_t row, int rank, int ranks, float scale,
                                       uint4 (&out)[TERMS]) {
    float f[8] = {};
    const float *p = a.v + row * a.v_stride + rank;
    if (rank < ranks) {
        for (int s = 0; s < a.splits; ++s) {
            const float4 u = *reinterpret_cast<const float4 *>(p), v = *reinterpret_cast<const float4 *>(p + 4);
            f[0] += u.x; f[1] += u.y; f[2] += u.z; f[3] += u.w;
            f[4] += v.x; f[5] += v.y; f[6] += v.z; f[7] += v.w;
            p += (int64_t)a.M * a.v_stride;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = rank + i < ranks ? f[i] * scale : 0.0f;
#pragma unroll
    for (int q = 0; q < TERMS; ++q) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[i] = bf16_pair(f[2 * i], f[2 * i + 1]);
            f[2 * i] -= bf16_lo(o[i]);
            f[2 * i + 1] -= bf16_hi(o[i]);
        }
        out[q] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// y of one tile for column runs of 64 per wave.  D[column][row] from B rows
// and v.  The rows of a wave's four column tiles are dealt so that each lane
// ends with 16 consecutive columns of its row.
template <int CT, int RK, bool F32, bool SORTED>
__global__ __launch_bounds__(256) void expand_kernel(LoraLaunch a) {
    constexpr int TERMS = F32 ? 3 : 2;
    __shared__ int member[16 * CT];
    const Tile t = find_tile<CT, SORTED>(a, blockIdx.y, member);
    if (t.count == 0) return;
    const int ranks = rank_of(a, t.adapter);
    if (ranks == 0 && a.base == a.y) return;   // these rows are already there
    const float scale = a.scales && t.adapter < a.adapters ? a.scales[t.adapter] : 1.0f;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int c16 = lane & 15, kg = lane >> 4;
    const int chunks = (ranks + 32 * RK - 1) / (32 * RK);
    int row[CT];
    uint4 vf[CT][RK][TERMS];
    auto load_chunk = [&](int ch) {
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            const int i = c * 16 + c16 < t.count ? c * 16 + c16 : 0;
            const int64_t at = t.v0 >= 0 ? t.v0 + i : member[i];
#pragma unroll
            for (int q = 0; q < RK; ++q)
                load_v<TERMS>(a, at, (ch * RK + q) * 32 + kg * 8, ranks, scale, vf[c][q]);
        }
    };
#pragma unroll
    for (int c = 0; c < CT; ++c) row[c] = c * 16 + c16 < t.count ? member[c * 16 + c16] : -1;
    if (chunks == 1) load_chunk(0);
    const int n_end = min(a.N, (int)(blockIdx.x + 1) * a.n_chunk);
    for (int n0 = blockIdx.x * a.n_chunk + w * 64; n0 < n_end; n0 += 256) {
        v4f acc[CT][4] = {};
        for (int ch = 0; ch < chunks; ++ch) {
            if (chunks > 1) load_chunk(ch);
            uint4 bv[4][RK];
#pragma unroll
            for (int q = 0; q < RK; ++q) {
                const int rank = (ch * RK + q) * 32 + kg * 8;
                // ranks past the adapter's: whatever B holds there is cleared
                uint32_t keep[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    keep[i] = (rank + 2 * i < ranks ? 0xFFFFu : 0u) | (rank + 2 * i + 1 < ranks ? 0xFFFF0000u : 0u);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n = min(n0 + (c16 >> 2) * 16 + j * 4 + (c16 & 3), a.N - 1);
                    uint4 b = make_uint4(0, 0, 0, 0);
                    if (rank < ranks)
                        b = *reinterpret_cast<const uint4 *>(a.B + ((int64_t)t.adapter * a.N + n) * a.max_rank + rank);
                    bv[j][q] = make_uint4(b.x & keep[0], b.y & keep[1], b.z & keep[2], b.w & keep[3]);
                }
            }
#pragma unroll
            for (int q = 0; q < RK; ++q)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int c = 0; c < CT; ++c)
#pragma unroll
                        for (int e = TERMS - 1; e >= 0; --e) acc[c][j] = mfma_bf16(bv[j][q], vf[c][q][e], acc[c][j]);
        }
        const int n = n0 + kg * 16;
        if (n >= n_end) continue;   // N and n_chunk are multiples of 16
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            if (row[c] < 0) continue;
            const int64_t at = (int64_t)row[c] * a.ldy + n, bt = (int64_t)row[c] * a.ldb + n;
            if constexpr (F32) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v4f o = acc[c][j];
                    if (a.base) o += *reinterpret_cast<const v4f *>(static_cast<const float *>(a.base) + bt + 4 * j);
                    *reinterpret_cast<v4f *>(static_cast<float *>(a.y) + at + 4 * j) = o;
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint4 b = make_uint4(0, 0, 0, 0);
                    if (a.base)
                        b = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.base) + bt + 8 * h);
                    const v4f p = acc[c][2 * h], q = acc[c][2 * h + 1];
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.y) + at + 8 * h) =
                        make_uint4(bf16_pair(bf16_lo(b.x) + p[0], bf16_hi(b.x) + p[1]),
                                   bf16_pair(bf16_lo(b.y) + p[2], bf16_hi(b.y) + p[3]),
                                   bf16_pair(bf16_lo(b.z) + q[0], bf16_hi(b.z) + q[1]),
                                   bf16_pair(bf16_lo(b.w) + q[2], bf16_hi(b.w) + q[3]));
                }
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

// Rows up to which a workgroup finds its tile by a ballot over the ids.
constexpr int kLoraDirectRows = 64;

void lora_plan(int M, int N, int K, int adapters, int max_rank, LoraPlan *p) {
    p->sorted = M > kLoraDirectRows;
    p->ct = M >= 1024 ? 4 : 1;
    const int tile_rows = 16 * p->ct;
    p->max_tiles = p->sorted ? (M + tile_rows - 1) / tile_rows + (adapters + 1 < M ? adapters + 1 : M) : M;
    p->rt = max_rank <= 16 ? 1 : max_rank <= 32 ? 2 : 4;
    p->rank_chunks = (max_rank + 16 * p->rt - 1) / (16 * p->rt);
    p->v_stride = (max_rank + 15) / 16 * 16;
    // K parts: enough workgroups to fill the GPU twice, with two steps of 32
    // or more for each of a workgroup's four waves
    const int steps = (K + 31) / 32;
    const int tiles = (M + tile_rows - 1) / tile_rows;
    int splits = 512 / ((p->sorted ? tiles : M) * p->rank_chunks);
    splits = splits > 16 ? 16 : splits < 1 ? 1 : splits;
    if (splits > steps / 8) splits = steps / 8 > 0 ? steps / 8 : 1;
    p->k_steps = (steps + 4 * splits - 1) / (4 * splits);
    p->splits = (steps + 4 * p->k_steps - 1) / (4 * p->k_steps);
    // columns per expand workgroup
    int n_chunk = 256;
    while ((int64_t)((N + n_chunk - 1) / n_chunk) * tiles > 2048 && n_chunk < 4096) n_chunk *= 2;
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
static void launch_shrink(const LoraPlan &p, const LoraLaunch &a, const dim3 &grid, hipStream_t s) {
    if (p.sorted) hipLaunchKernelGGL((shrink_kernel<CT, RT, true>), grid, dim3(256), 0, s, a);
    else if constexpr (CT == 1) hipLaunchKernelGGL((shrink_kernel<CT, RT, false>), grid, dim3(256), 0, s, a);
}

template <int CT, int RK>
static void launch_expand(const LoraPlan &p, bool f32, const LoraLaunch &a, const dim3 &grid, hipStream_t s) {
    if (p.sorted) {
        if (f32) hipLaunchKernelGGL((expand_kernel<CT, RK, true, true>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((expand_kernel<CT, RK, false, true>), grid, dim3(256), 0, s, a);
    } else if constexpr (CT == 1) {
        if (f32) hipLaunchKernelGGL((expand_kernel<CT, RK, true, false>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((expand_kernel<CT, RK, false, false>), grid, dim3(256), 0, s, a);
    }
}

hipError_t launch_lora(const LoraPlan &p, bool f32, const LoraLaunch &a, hipStream_t s) {
    hipError_t e;
    if (p.sorted) {
        hipLaunchKernelGGL(group_kernel, dim3(1), dim3(1024), 0, s, a, 16 * p.ct);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const dim3 sg(p.splits, p.max_tiles, p.rank_chunks);
    if (p.ct == 1) {
        if (p.rt == 1) launch_shrink<1, 1>(p, a, sg, s);
        else if (p.rt == 2) launch_shrink<1, 2>(p, a, sg, s);
        else launch_shrink<1, 4>(p, a, sg, s);
    } else {
        if (p.rt == 1) launch_shrink<4, 1>(p, a, sg, s);
        else if (p.rt == 2) launch_shrink<4, 2>(p, a, sg, s);
        else launch_shrink<4, 4>(p, a, sg, s);
    }
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 eg((a.N + p.n_chunk - 1) / p.n_chunk, p.max_tiles);
    if (p.ct == 1) {
        if (p.rt <= 2) launch_expand<1, 1>(p, f32, a, eg, s);
        else launch_expand<1, 2>(p, f32, a, eg, s);
    } else {
        if (p.rt <= 2) launch_expand<4, 1>(p, f32, a, eg, s);
        else launch_expand<4, 2>(p, f32, a, eg, s);
    }
    return hipGetLastError();
}

}  // namespace qlin
