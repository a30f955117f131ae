// qlin_expert_rows.hip -- the way of the tokens' rows into the grouped product
// (quantize and scatter) and back out of it (weighted gather).
#include "qlin_device.h"

namespace qlin {

namespace {

// ------------------------------------------------------------------ dispatch

typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// Eight codes of a row.  Non-temporal: topk rows are written for each that is
// read, 15.1 us against 17.0 for 4096 tokens of 2048 to 8 rows each.
__device__ __forceinline__ void store_codes(uint8_t *to, uint2 q) {
    __builtin_nontemporal_store(v2u{q.x, q.y}, reinterpret_cast<v2u *>(to));
}

// One token per workgroup: the row is read once, quantized as
// quant_token_kernel does, and its codes go to each of the token's rows.
// CPT as there.
template <int FMT, int CPT>
__global__ __launch_bounds__(256) void dispatch_token_kernel(DispatchLaunch a) {
    __shared__ float red[4];
    const int t = blockIdx.x, tid = threadIdx.x;
    const uint16_t *row = a.x + (int64_t)t * a.ldx;
    const int nch = a.K >> 3;
    float amax = 0.0f;
    uint4 v[CPT > 0 ? CPT : 1];
    if constexpr (CPT > 0) {
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            const int c = tid + j * 256;
            v[j] = c < nch ? *reinterpret_cast<const uint4 *>(row + c * 8) : make_uint4(0, 0, 0, 0);
            amax = fmaxf(amax, absmax8(v[j]));
        }
    } else {
        for (int c = tid; c < nch; c += 256)
            amax = fmaxf(amax, absmax8(*reinterpret_cast<const uint4 *>(row + c * 8)));
    }
    amax = wave_max(amax);
    if ((tid & 63) == 0) red[tid >> 6] = amax;
    __syncthreads();
    amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float s = amax == 0.0f ? 0.0f : amax / qmax_of<FMT>();
    const float y = recip_scale(s);
    const int *slots = a.slots + (int64_t)t * a.topk;
    auto store = [&](int c, uint4 chunk) {
        const uint2 q = quant8<FMT>(chunk, s, y);
        for (int j = 0; j < a.topk; ++j) {
            const int slot = slots[j];
            if ((unsigned)slot < (unsigned)a.total_rows)
                store_codes(a.xq + (int64_t)slot * a.K + c * 8, q);
        }
    };
    if constexpr (CPT > 0) {
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            const int c = tid + j * 256;
            if (c < nch) store(c, v[j]);
        }
    } else {
        for (int c = tid; c < nch; c += 256) store(c, *reinterpret_cast<const uint4 *>(row + c * 8));
    }
    if (tid < a.topk && (unsigned)slots[tid] < (unsigned)a.total_rows) a.xs[slots[tid]] = s;
}

// 1x128 groups: 16 lanes own one (token, group), as quant_group_kernel.
__global__ __launch_bounds__(256) void dispatch_group_kernel(DispatchLaunch a) {
    const int G = a.K / kGroup;
    const int64_t gi = blockIdx.x * (int64_t)16 + (threadIdx.x >> 4);
    const int j = threadIdx.x & 15;
    const bool live = gi < (int64_t)a.T * G;
    const int t = live ? (int)(gi / G) : 0;
    const int g = live ? (int)(gi - (int64_t)t * G) : 0;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (live) v = *reinterpret_cast<const uint4 *>(a.x + (int64_t)t * a.ldx + g * kGroup + j * 8);
    const float amax = row16_max(absmax8(v));
    const float s = amax == 0.0f ? 0.0f : amax / 448.0f;
    if (!live) return;
    const uint2 q = quant8<FMT_BLOCK>(v, s, recip_scale(s));
    for (int i = 0; i < a.topk; ++i) {
        const int slot = a.slots[(int64_t)t * a.topk + i];
        if ((unsigned)slot >= (unsigned)a.total_rows) continue;
        store_codes(a.xq + (int64_t)slot * a.K + g * kGroup + j * 8, q);
        if (j == 0) a.xs[(int64_t)slot * G + g] = s;
    }
}

// ------------------------------------------------------------------- combine

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// two fp32 -> two bf16, nearest even, NaN kept
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    v2bf p;
    p[0] = (__bf16)lo;
    p[1] = (__bf16)hi;
    return __builtin_bit_cast(uint32_t, p);
}

// Eight elements at p as fp32, and back.  Every one of them is read or written
// once: with the non-temporal policy on both, 4096 tokens of 2048 from 8 bf16
// rows each and a residual take 27.5 us against 35 (6.1 TB/s).
template <bool F32>
__device__ __forceinline__ void load8(const void *base, int64_t at, float (&f)[8]) {
    if constexpr (F32) {
        const v4f *p = reinterpret_cast<const v4f *>(static_cast<const float *>(base) + at);
        const v4f u = __builtin_nontemporal_load(p), v = __builtin_nontemporal_load(p + 1);
        f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
        f[4] = v.x; f[5] = v.y; f[6] = v.z; f[7] = v.w;
    } else {
        const v4u u =
            __builtin_nontemporal_load(reinterpret_cast<const v4u *>(static_cast<const uint16_t *>(base) + at));
        const uint32_t q[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(q[i]);
            f[2 * i + 1] = bf16_hi(q[i]);
        }
    }
}
template <bool F32>
__device__ __forceinline__ void store8(void *base, int64_t at, const float (&f)[8]) {
    if constexpr (F32) {
        v4f *p = reinterpret_cast<v4f *>(static_cast<float *>(base) + at);
        __builtin_nontemporal_store(v4f{f[0], f[1], f[2], f[3]}, p);
        __builtin_nontemporal_store(v4f{f[4], f[5], f[6], f[7]}, p + 1);
    } else {
        const v4u o = {bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7])};
        __builtin_nontemporal_store(o, reinterpret_cast<v4u *>(static_cast<uint16_t *>(base) + at));
    }
}

// Eight columns of one token per thread.
template <bool H32, bool Y32>
__global__ __launch_bounds__(256) void combine_kernel(CombineLaunch a) {
    const int n = (blockIdx.x * 256 + threadIdx.x) * 8;
    const int t = blockIdx.y;
    if (n >= a.N) return;
    float acc[8] = {};
    for (int j = 0; j < a.topk; ++j) {
        const int slot = a.slots[(int64_t)t * a.topk + j];
        if ((unsigned)slot >= (unsigned)a.total_rows) continue;
        const float w = a.weights[(int64_t)t * a.topk + j];
        float h[8];
        load8<H32>(a.h, (int64_t)slot * a.ldh + n, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(w, h[i], acc[i]);
    }
    if (a.add) {
        float r[8];
        load8<Y32>(a.add, (int64_t)t * a.ldadd + n, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += r[i];
    }
    store8<Y32>(a.y, (int64_t)t * a.ldy + n, acc);
}

}  // namespace

// --------------------------------------------------------------- launchers

template <int FMT>
static void launch_dispatch_token(const DispatchLaunch &a, hipStream_t s) {
    const dim3 grid(a.T), block(256);
    const int cpt = (a.K / 8 + 255) / 256;
    if (cpt <= 1) hipLaunchKernelGGL((dispatch_token_kernel<FMT, 1>), grid, block, 0, s, a);
    else if (cpt <= 2) hipLaunchKernelGGL((dispatch_token_kernel<FMT, 2>), grid, block, 0, s, a);
    else if (cpt <= 4) hipLaunchKernelGGL((dispatch_token_kernel<FMT, 4>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((dispatch_token_kernel<FMT, 0>), grid, block, 0, s, a);
}

hipError_t launch_dispatch(int fmt, const DispatchLaunch &a, hipStream_t s) {
    if (fmt == FMT_BLOCK) {
        // a launch has fewer than 2^32 threads, 16 for each group
        const int G = a.K / kGroup, most = (1 << 27) / G;
        for (int t0 = 0; t0 < a.T; t0 += most) {
            DispatchLaunch c = a;
            c.T = a.T - t0 < most ? a.T - t0 : most;
            c.x += (int64_t)t0 * a.ldx;
            c.slots += (int64_t)t0 * a.topk;
            const int64_t groups = (int64_t)c.T * G;
            hipLaunchKernelGGL(dispatch_group_kernel, dim3((unsigned)((groups + 15) / 16)), dim3(256), 0, s, c);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    }
    if (fmt == FMT_I8) {
        launch_dispatch_token<FMT_I8>(a, s);
    } else {
        launch_dispatch_token<FMT_FP8>(a, s);
    }
    return hipGetLastError();
}

hipError_t launch_combine(bool h32, bool y32, const CombineLaunch &a, hipStream_t s) {
    const dim3 block(256);
    // tokens fill grid y, in launches of at most 65535
    for (int t0 = 0; t0 < a.T; t0 += 65535) {
        CombineLaunch c = a;
        c.T = a.T - t0 < 65535 ? a.T - t0 : 65535;
        c.slots += (int64_t)t0 * a.topk;
        c.weights += (int64_t)t0 * a.topk;
        c.y = static_cast<char *>(a.y) + (int64_t)t0 * a.ldy * (y32 ? 4 : 2);
        if (a.add) c.add = static_cast<const char *>(a.add) + (int64_t)t0 * a.ldadd * (y32 ? 4 : 2);
        const dim3 grid((a.N / 8 + 255) / 256, c.T);
        if (h32 && y32) hipLaunchKernelGGL((combine_kernel<true, true>), grid, block, 0, s, c);
        else if (h32) hipLaunchKernelGGL((combine_kernel<true, false>), grid, block, 0, s, c);
        else if (y32) hipLaunchKernelGGL((combine_kernel<false, true>), grid, block, 0, s, c);
        else hipLaunchKernelGGL((combine_kernel<false, false>), grid, block, 0, s, c);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace qlin
