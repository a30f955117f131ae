// qlin_cache.hip -- keys and values into a paged 8-bit cache with one scale for
// each page and head, and back out of it.
//
// One workgroup (or, for few tokens, one wave) has one page and head of keys or of
// values, so the page's scale needs no exchange between workgroups, and a call is one
// launch.  Rows are read and written 16 consecutive bytes a lane; the tiles' order of
// bytes (include/qlin.h) is made in the LDS.  Bytes bound the large calls: prompts of
// 11489 tokens (8 heads of 128, bf16, 70 MB) are stored in 23 us, 42974 tokens (264
// MB) read back in 50.4, 5.2 TB/s; 63 without the non-temporal policy on what is
// written, which nobody reads soon.  Small calls are a chain of dependent loads: offsets
// and lengths, the page, its scale, 5.0 us with the launch.
#include "qlin_sequences.h"

namespace qlin {

namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kTile = 16;                    // tokens of a tile
constexpr int kRowPad = 16;                  // bytes behind each LDS row of codes
// Tokens a sequence, on average, up to which a wave has a page and head, not a
// workgroup.  32 sequences, us a call: 8 tokens each 5.0 and 5.0, 16 tokens 5.6 and 4.9,
// 64 tokens 17.5 and 8.0; 256 sequences of one token 5.7 and 16.3.  The host knows counts alone, so a
// long prompt beside many slots without tokens is the waves' too: one of 2000 tokens in 251 slots, 8
// heads of 128, pages of 64, 19.8 us where workgroups take 13.5; 8 of 256, pages of 128, 94 and 31.
// (A wave with eight loads on their way, 21.8 and 69; long pages by four waves together through
// the LDS, 19.8 and 53, but 512 sequences of one token with pages of 128 then take 16.6 for 9.8.)
constexpr int kFewTokens = 8;

// four codes of a word as fp32
template <int FMT>
__device__ __forceinline__ v4f code_values(uint32_t w) {
    if constexpr (FMT == FMT_I8)
        return v4f{(float)(int8_t)w, (float)(int8_t)(w >> 8), (float)(int8_t)(w >> 16), (float)(int8_t)(w >> 24)};
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    return v4f{lo[0], lo[1], hi[0], hi[1]};
}

// the codes of four values, given their scale and y = 1 / s (quant8's steps:
// the quotients are the IEEE ones)
template <int FMT>
__device__ __forceinline__ uint32_t quant4(v4f x, float s, float y) {
    uint32_t out = 0;
    if (!(s >= kFastScaleMin)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) out |= quant_code<FMT>(x[i], s) << (8 * i);
        return out;
    }
    float t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float q = div_by_scale(fabsf(x[i]), s, y);
        if constexpr (FMT == FMT_I8) q = __builtin_rintf(fminf(q, 127.0f));
        else q = fminf(q, 448.0f);
        t[i] = __builtin_copysignf(q, x[i]);
    }
    if constexpr (FMT == FMT_I8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) out |= ((uint32_t)(int32_t)t[i] & 0xFFu) << (8 * i);
        return out;
    }
    const int pk = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], pk, true);
}

// four codes under a scale that grew from `was` to s
template <int FMT>
__device__ __forceinline__ uint32_t requant4(uint32_t w, float was, float s, float y) {
    v4f x = code_values<FMT>(w);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] *= was;
    return quant4<FMT>(x, s, y);
}

// bytes (row, column) of four words -> (column, row)
__device__ __forceinline__ uint4 transposed(uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
    const uint32_t a = __builtin_amdgcn_perm(r1, r0, 0x05010400u), b = __builtin_amdgcn_perm(r1, r0, 0x07030602u);
    const uint32_t c = __builtin_amdgcn_perm(r3, r2, 0x05010400u), d = __builtin_amdgcn_perm(r3, r2, 0x07030602u);
    return make_uint4(__builtin_amdgcn_perm(c, a, 0x05040100u), __builtin_amdgcn_perm(c, a, 0x07060302u),
                      __builtin_amdgcn_perm(d, b, 0x05040100u), __builtin_amdgcn_perm(d, b, 0x07060302u));
}

// What a workgroup has: a page and head, and the call's tokens in it.
struct PageWork {
    int page;          // of the pool; -1: nothing to do
    int had;           // the page's tokens before the call's first in it
    int n;             // the call's tokens in it
    int row;           // row of the first in the call's tensors
};

__device__ __forceinline__ PageWork page_work(const CacheArgs &c) {
    PageWork w = {-1, 0, 0, 0};
    int within, first;
    const int s = unit_sequence(
        c, blockIdx.x, [&](const Sequence &q) { int f; return touched_pages(c, q, &f); }, &within);
    if (s < 0) return w;
    const Sequence q = sequence_at(c, s);
    touched_pages(c, q, &first);
    const int page = first + within;
    const int lo = max(q.start, page << c.page_shift);
    w.page = pool_page(c, s, page);
    w.had = lo - (page << c.page_shift);
    w.n = (int)min((int64_t)q.length, (int64_t)(page + 1) << c.page_shift) - lo;
    w.row = q.first + lo - q.start;
    return w;
}

template <bool F32>
__device__ __forceinline__ void load_row8(const void *base, int64_t at, v4f *x) {
    if constexpr (F32) {
        const v4f *p = reinterpret_cast<const v4f *>(static_cast<const float *>(base) + at);
        x[0] = p[0];
        x[1] = p[1];
    } else {
        const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + at);
        x[0] = v4f{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
        x[1] = v4f{bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w)};
    }
}

// log2 of the lanes that a row of D / 8 pieces of 8 channels takes
__host__ __device__ __forceinline__ int row_lanes_shift(int D) { return D <= 64 ? 3 : D <= 128 ? 4 : 5; }

// NI: passes of the workgroup over a full page's rows; the rows stay in
// registers between their maximum and their codes.
template <int FMT, bool F32, int NI>
__global__ __launch_bounds__(256) void append_kernel(RowsLaunch a, int D) {
    extern __shared__ uint4 lds[];
    __shared__ float red[4];
    uint8_t *const codes = reinterpret_cast<uint8_t *>(lds);     // [tokens][D + kRowPad]
    const CacheArgs &c = a.c;
    const int stride = D + kRowPad, tid = threadIdx.x;
    const int head = blockIdx.y >> 1;
    const bool values = blockIdx.y & 1;
    const PageWork w = page_work(c);
    if (w.page < 0) return;
    const int64_t slot = (int64_t)w.page * c.heads + head;
    float *const scale_at = (values ? c.v_scales : c.k_scales) + slot;
    const float was = w.had > 0 ? *scale_at : 0.0f;

    const int shift = row_lanes_shift(D), ch = (tid & ((1 << shift) - 1)) * 8, row0 = tid >> shift, rows = 256 >> shift;
    const void *src = values ? a.v : a.k;
    const int64_t ld = values ? a.ldv : a.ldk;
    v4f x[NI][2];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int r = row0 + i * rows;
        x[i][0] = x[i][1] = v4f{0, 0, 0, 0};
        if (r < w.n && ch < D) load_row8<F32>(src, (int64_t)(w.row + r) * ld + (int64_t)head * D + ch, x[i]);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[i][e >> 2][e & 3]));
    amax = wave_max(amax);
    if ((tid & 63) == 0) red[tid >> 6] = amax;
    __syncthreads();
    amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float now = fmaxf(was, amax / qmax_of<FMT>());
    const float y = recip_scale(now);
    const bool grown = now > was && w.had > 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int r = row0 + i * rows;
        if (r < w.n && ch < D)
            *reinterpret_cast<uint2 *>(codes + r * stride + ch) =
                make_uint2(quant4<FMT>(x[i][0], now, y), quant4<FMT>(x[i][1], now, y));
    }
    __syncthreads();
    if (tid == 0) *scale_at = now;

    // tiles: all that hold tokens where the older codes change, else the new tokens'
    const int end = w.had + w.n;
    const int tile0 = grown ? 0 : w.had / kTile, tiles = (end + kTile - 1) / kTile - tile0;
    const int J = D / 64;
    const int64_t base = slot * ((int64_t)D << c.page_shift) + (int64_t)tile0 * kTile * D;
    if (!values) {
        uint4 *const out = reinterpret_cast<uint4 *>(c.k + base);
        for (int p = tid; p < tiles * D; p += 256) {
            const int block = p >> 6, tile = block / J, j = block - tile * J;
            const int t = (tile0 + tile) * kTile + (p & 15), d = 64 * j + 16 * ((p >> 4) & 3);
            if (t >= w.had && t < end) {
                out[p] = *reinterpret_cast<const uint4 *>(codes + (t - w.had) * stride + d);
            } else if (grown && t < w.had) {
                const uint4 o = out[p];
                out[p] = make_uint4(requant4<FMT>(o.x, was, now, y), requant4<FMT>(o.y, was, now, y),
                                    requant4<FMT>(o.z, was, now, y), requant4<FMT>(o.w, was, now, y));
            }
        }
    } else {
        // four pieces of 16 bytes at a time: 4 tokens, of each 4 channels in every 16
        uint4 *const out = reinterpret_cast<uint4 *>(c.v + base);
        for (int p = tid; p < tiles * D / 4; p += 256) {
            const int block = p >> 4, tile = block / J, j = block - tile * J;
            const int t0 = (tile0 + tile) * kTile + 4 * ((p >> 2) & 3), d = 64 * j + 4 * (p & 3);
            if (t0 >= end || (!grown && t0 + 4 <= w.had)) continue;
            uint32_t fresh = 0, older = 0;       // bytes of the new tokens, and of those quantized again
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t byte = 0xFFu << (8 * i);
                if (t0 + i >= w.had && t0 + i < end) fresh |= byte;
                if (grown && t0 + i < w.had) older |= byte;
            }
            uint32_t o[4][4];                    // [channel][16s of channels]
            if (fresh != 0xFFFFFFFFu) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 v = out[4 * p + i];
                    o[i][0] = v.x; o[i][1] = v.y; o[i][2] = v.z; o[i][3] = v.w;
                }
                if (older) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        uint32_t &v = o[i >> 2][i & 3];
                        v = (v & ~older) | (requant4<FMT>(v, was, now, y) & older);
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                uint32_t r[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = min(max(t0 + i - w.had, 0), w.n - 1);      // a row that is there
                    r[i] = *reinterpret_cast<const uint32_t *>(codes + t * stride + d + 16 * b);
                }
                const uint4 v = transposed(r[0], r[1], r[2], r[3]);
                const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[i][b] = fresh == 0xFFFFFFFFu ? q[i] : (o[i][b] & ~fresh) | (q[i] & fresh);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) out[4 * p + i] = make_uint4(o[i][0], o[i][1], o[i][2], o[i][3]);
        }
    }
}

// The same for few tokens a sequence: a wave has a page and head of keys or of
// values, and nothing is exchanged.  A lane's eight codes go straight to their places:
// eight bytes of a key's row, or eight single bytes of values.  Older codes that
// change are written before them, by the same wave.
template <int FMT, bool F32>
__global__ __launch_bounds__(256) void append_few_kernel(RowsLaunch a, int D) {
    constexpr int NI = 2;                        // passes whose rows stay in registers
    const CacheArgs &c = a.c;
    const int lane = threadIdx.x & 63;
    const int item = blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), head = item >> 1;
    const bool values = item & 1;
    if (head >= c.heads) return;
    const PageWork w = page_work(c);
    if (w.page < 0) return;
    const int64_t slot = (int64_t)w.page * c.heads + head;
    float *const scale_at = (values ? c.v_scales : c.k_scales) + slot;
    uint8_t *const page = (values ? c.v : c.k) + slot * ((int64_t)D << c.page_shift);
    const int shift = row_lanes_shift(D), ch = (lane & ((1 << shift) - 1)) * 8, row0 = lane >> shift, rows = 64 >> shift;
    const void *src = values ? a.v : a.k;
    const int64_t at = (int64_t)(w.row + row0) * (values ? a.ldv : a.ldk) + (int64_t)head * D + ch;
    const int64_t step = (values ? a.ldv : a.ldk) * rows;
    const bool live = ch < D;
    v4f x[NI][2];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        x[i][0] = x[i][1] = v4f{0, 0, 0, 0};
        if (row0 + i * rows < w.n && live) load_row8<F32>(src, at + i * step, x[i]);
    }
    const float was = w.had > 0 ? *scale_at : 0.0f;
    auto most = [](const v4f (&v)[2]) {
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[e >> 2][e & 3]));
        return m;
    };
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) amax = fmaxf(amax, most(x[i]));
    for (int i = NI; i * rows < w.n; ++i) {
        v4f more[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
        if (row0 + i * rows < w.n && live) load_row8<F32>(src, at + i * step, more);
        amax = fmaxf(amax, most(more));
    }
    amax = wave_max(amax);
    const float now = fmaxf(was, amax / qmax_of<FMT>());
    const float y = recip_scale(now);
    if (w.had > 0 && now > was) {
        // pieces of 16 bytes: a key's 16 channels, or four tokens of four channels of values
        uint4 *const pieces = reinterpret_cast<uint4 *>(page);
        const int J = D / 64, tiles = (w.had + kTile - 1) / kTile;
        for (int p = lane; p < tiles * D; p += 64) {
            const int first = (p >> 6) / J * kTile + (values ? 4 * ((p >> 4) & 3) : p & 15);
            if (first >= w.had) continue;
            uint32_t older = 0xFFFFFFFFu;
            if (values && first + 4 > w.had) older = 0xFFFFFFFFu >> (8 * (first + 4 - w.had));
            const uint4 o = pieces[p];
            auto again = [&](uint32_t v) { return (v & ~older) | (requant4<FMT>(v, was, now, y) & older); };
            pieces[p] = make_uint4(again(o.x), again(o.y), again(o.z), again(o.w));
        }
        __threadfence_block();                   // before other lanes store new tokens into the same pieces
    }
    if (lane == 0) *scale_at = now;
    auto store = [&](int r, const v4f (&v)[2]) {
        const int t = w.had + r, d = ch;
        const uint2 q = make_uint2(quant4<FMT>(v[0], now, y), quant4<FMT>(v[1], now, y));
        uint8_t *to = page + (t / kTile) * (kTile * D) + 1024 * (d / 64);
        if (!values) {
            *reinterpret_cast<uint2 *>(to + 256 * (d % 64 / 16) + 16 * (t % kTile) + d % 16) = q;
        } else {
            to += 256 * (t % kTile / 4) + 16 * (d % 16) + 4 * (d % 64 / 16) + t % 4;
#pragma unroll
            for (int e = 0; e < 8; ++e) to[16 * e] = (uint8_t)((e < 4 ? q.x : q.y) >> (8 * (e & 3)));
        }
    };
#pragma unroll
    for (int i = 0; i < NI; ++i)
        if (row0 + i * rows < w.n && live) store(row0 + i * rows, x[i]);
    for (int i = NI; row0 + i * rows < w.n && live; ++i) {
        v4f more[2];
        load_row8<F32>(src, at + i * step, more);
        store(row0 + i * rows, more);
    }
}

template <int FMT, bool F32>
__global__ __launch_bounds__(256) void read_kernel(RowsLaunch a, int D) {
    extern __shared__ uint4 lds[];
    uint8_t *const codes = reinterpret_cast<uint8_t *>(lds);
    const CacheArgs &c = a.c;
    const int stride = D + kRowPad, tid = threadIdx.x;
    const int head = blockIdx.y >> 1;
    const bool values = blockIdx.y & 1;
    void *dst = values ? a.v : a.k;
    if (!dst) return;
    const PageWork w = page_work(c);
    if (w.page < 0) return;
    const int64_t slot = (int64_t)w.page * c.heads + head;
    const float scale = (values ? c.v_scales : c.k_scales)[slot];
    const int end = w.had + w.n, tile0 = w.had / kTile, tiles = (end + kTile - 1) / kTile - tile0, J = D / 64;
    const uint4 *src = reinterpret_cast<const uint4 *>((values ? c.v : c.k) + slot * ((int64_t)D << c.page_shift) +
                                                       (int64_t)tile0 * kTile * D);
    if (!values) {
        for (int p = tid; p < tiles * D; p += 256) {
            const int block = p >> 6, tile = block / J, j = block - tile * J;
            *reinterpret_cast<uint4 *>(codes + (tile * kTile + (p & 15)) * stride + 64 * j + 16 * ((p >> 4) & 3)) = src[p];
        }
    } else {
        for (int p = tid; p < tiles * D / 4; p += 256) {
            const int block = p >> 4, tile = block / J, j = block - tile * J;
            const uint4 o0 = src[4 * p], o1 = src[4 * p + 1], o2 = src[4 * p + 2], o3 = src[4 * p + 3];
            uint8_t *to = codes + (tile * kTile + 4 * ((p >> 2) & 3)) * stride + 64 * j + 4 * (p & 3);
            const uint4 r[4] = {transposed(o0.x, o1.x, o2.x, o3.x), transposed(o0.y, o1.y, o2.y, o3.y),
                                transposed(o0.z, o1.z, o2.z, o3.z), transposed(o0.w, o1.w, o2.w, o3.w)};
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                *reinterpret_cast<uint32_t *>(to + 16 * b) = r[b].x;
                *reinterpret_cast<uint32_t *>(to + stride + 16 * b) = r[b].y;
                *reinterpret_cast<uint32_t *>(to + 2 * stride + 16 * b) = r[b].z;
                *reinterpret_cast<uint32_t *>(to + 3 * stride + 16 * b) = r[b].w;
            }
        }
    }
    __syncthreads();
    const int shift = row_lanes_shift(D), ch = (tid & ((1 << shift) - 1)) * 8, rows = 256 >> shift;
    const int64_t ld = values ? a.ldv : a.ldk;
    if (ch >= D) return;
    for (int r = tid >> shift; r < w.n; r += rows) {
        const uint2 q = *reinterpret_cast<const uint2 *>(codes + (r + w.had - tile0 * kTile) * stride + ch);
        v4f x = code_values<FMT>(q.x), z = code_values<FMT>(q.y);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] *= scale;
            z[i] *= scale;
        }
        const int64_t at = (int64_t)(w.row + r) * ld + (int64_t)head * D + ch;
        if constexpr (F32) {
            v4f *to = reinterpret_cast<v4f *>(static_cast<float *>(dst) + at);
            __builtin_nontemporal_store(x, to);
            __builtin_nontemporal_store(z, to + 1);
        } else {
            const v4u b = {bf16_bits(x[0]) | (bf16_bits(x[1]) << 16), bf16_bits(x[2]) | (bf16_bits(x[3]) << 16),
                           bf16_bits(z[0]) | (bf16_bits(z[1]) << 16), bf16_bits(z[2]) | (bf16_bits(z[3]) << 16)};
            __builtin_nontemporal_store(b, reinterpret_cast<v4u *>(static_cast<uint16_t *>(dst) + at));
        }
    }
}

size_t page_lds(const CacheArgs &c, int D) { return (size_t)(D + kRowPad) << c.page_shift; }

template <int FMT, bool F32>
void launch_append_t(int D, const RowsLaunch &a, hipStream_t s) {
    const dim3 block(256);
    if (a.c.T <= kFewTokens * (int64_t)a.c.B) {
        hipLaunchKernelGGL((append_few_kernel<FMT, F32>), dim3(a.units, (2 * a.c.heads + 3) / 4), block, 0, s, a, D);
        return;
    }
    const int rows = 256 >> row_lanes_shift(D), passes = ((1 << a.c.page_shift) + rows - 1) / rows;
    const dim3 grid(a.units, 2 * a.c.heads);
    const size_t lds = page_lds(a.c, D);
#define QLIN_APPEND(NI) hipLaunchKernelGGL((append_kernel<FMT, F32, NI>), grid, block, lds, s, a, D)
    if (passes <= 1) QLIN_APPEND(1);
    else if (passes <= 2) QLIN_APPEND(2);
    else if (passes <= 4) QLIN_APPEND(4);
    else if (passes <= 8) QLIN_APPEND(8);
    else QLIN_APPEND(16);
#undef QLIN_APPEND
}

}  // namespace

// (sequence, touched page) pairs of a call, at most: each sequence with n tokens
// touches fewer than n / page + 2 pages, and at most n
int64_t cache_units(const CacheArgs &c) {
    const int64_t T = c.T, some = c.B < T ? c.B : T;
    const int64_t by_page = (T >> c.page_shift) + 2 * some;
    return by_page < T ? by_page : T;
}

hipError_t launch_append(int fmt, bool f32, int head_dim, const RowsLaunch &a, hipStream_t s) {
    if (fmt == FMT_I8) f32 ? launch_append_t<FMT_I8, true>(head_dim, a, s) : launch_append_t<FMT_I8, false>(head_dim, a, s);
    else f32 ? launch_append_t<FMT_FP8, true>(head_dim, a, s) : launch_append_t<FMT_FP8, false>(head_dim, a, s);
    return hipGetLastError();
}

hipError_t launch_read(int fmt, bool f32, int head_dim, const RowsLaunch &a, hipStream_t s) {
    const dim3 grid(a.units, 2 * a.c.heads), block(256);
    const size_t lds = page_lds(a.c, head_dim);
    if (fmt == FMT_I8) {
        if (f32) hipLaunchKernelGGL((read_kernel<FMT_I8, true>), grid, block, lds, s, a, head_dim);
        else hipLaunchKernelGGL((read_kernel<FMT_I8, false>), grid, block, lds, s, a, head_dim);
    } else {
        if (f32) hipLaunchKernelGGL((read_kernel<FMT_FP8, true>), grid, block, lds, s, a, head_dim);
        else hipLaunchKernelGGL((read_kernel<FMT_FP8, false>), grid, block, lds, s, a, head_dim);
    }
    return hipGetLastError();
}

}  // namespace qlin
