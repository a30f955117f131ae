// qlin_route.hip -- routing tokens to experts (scores, top-k choice, weights,
// rows grouped by expert), and the way of the tokens' rows into the grouped
// product (quantize and scatter) and back out of it (weighted gather).
//
// The pages name MoE layers as the next target ("Building a High-Performance
// and Portable vLLM Linear Backend with Helion", section "Future work",
// model-coverage paragraph).
#include <type_traits>

#include "qlin_device.h"

namespace qlin {

namespace {

constexpr int kRouteWaves = 16;                   // waves of a routing workgroup
constexpr int kRouteThreads = 64 * kRouteWaves;
constexpr float kFltMax = 3.402823466e38f;

// ------------------------------------------------------------ wave reductions

// one DPP step of an unsigned maximum / a sum (see max_dpp)
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ uint32_t umax_dpp(uint32_t v) {
    const uint32_t moved = (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, ROW_MASK, 0xF, false);
    return v > moved ? v : moved;
}
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ float add_dpp(float v) {
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROW_MASK, 0xF, false));
}
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ double add_dpp(double v) {
    const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, ROW_MASK, 0xF, false);
    const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, ROW_MASK, 0xF, false);
    return v + __hiloint2double(hi, lo);
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
    v = umax_dpp<0xB1>(v);
    v = umax_dpp<0x4E>(v);
    v = umax_dpp<0x141>(v);
    v = umax_dpp<0x140>(v);
    v = umax_dpp<0x142, 0xA>(v);
    v = umax_dpp<0x143, 0xC>(v);
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint64_t wave_umax(uint64_t v) {
    const uint32_t hi = wave_umax((uint32_t)(v >> 32));
    const uint32_t lo = wave_umax((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return ((uint64_t)hi << 32) | lo;
}
template <typename F>
__device__ __forceinline__ F wave_sum_lane63(F v) {
    v = add_dpp<0xB1>(v);
    v = add_dpp<0x4E>(v);
    v = add_dpp<0x141>(v);
    v = add_dpp<0x140>(v);
    v = add_dpp<0x142, 0xA>(v);
    return add_dpp<0x143, 0xC>(v);
}
__device__ __forceinline__ float wave_sum(float v) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wave_sum_lane63(v)), 63));
}
__device__ __forceinline__ double wave_sum(double v) {
    v = wave_sum_lane63(v);
    return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), 63),
                            __builtin_amdgcn_readlane(__double2loint(v), 63));
}

// ------------------------------------------------------------- ordered keys

// Numbers as unsigned integers of the same order; -0 counts as +0.  No
// number but NaN (which never gets here) maps to 0: the key of what is closed.
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ uint64_t ordered(double f) {
    const uint64_t u = (uint64_t)__double_as_longlong(f + 0.0);
    return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double unordered(uint64_t k) {
    return __longlong_as_double((long long)(k >> 63 ? k ^ 0x8000000000000000ull : ~k));
}

// Lowest expert whose key is `best` (expert e = lane + 64 j): ballots in
// the order of j, then the lowest lane.
template <int EPL, typename Key>
__device__ __forceinline__ int first_with(const Key (&key)[EPL], Key best) {
    int at = -1;
#pragma unroll
    for (int j = EPL - 1; j >= 0; --j) {
        const uint64_t b = __ballot(key[j] == best);
        if (b) at = 64 * j + __ffsll((unsigned long long)b) - 1;
    }
    return at;
}

// One token, by one wave: lane j < topk ends with the j-th chosen expert (-1:
// none) and its weight.  Lane l holds experts l, l + 64, ...
template <int EPL, bool WIDE>
__device__ __forceinline__ void route_token(const RouteLaunch &a, int t, int lane, int &my_id, float &my_w) {
    using Key = std::conditional_t<WIDE, uint64_t, uint32_t>;
    float l[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = lane + 64 * j;
        l[j] = -INFINITY;
        if (e < a.experts) {
            const int64_t at = (int64_t)t * a.ld + e;
            l[j] = a.logits_bf16 ? __uint_as_float((uint32_t) static_cast<const uint16_t *>(a.logits)[at] << 16)
                                 : static_cast<const float *>(a.logits)[at];
        }
        if (l[j] != l[j]) l[j] = -INFINITY;
        l[j] = fminf(l[j], kFltMax);
    }
    float top = -INFINITY;
    if (a.score == QLIN_SCORE_SOFTMAX) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) top = fmaxf(top, l[j]);
        top = wave_max(top);
    }
    // the order of the choice
    Key key[EPL];
    if constexpr (WIDE) {
        double s[EPL];
        if (a.score == QLIN_SCORE_SOFTMAX) {
            double sum = 0.0;
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                s[j] = l[j] > -INFINITY ? exp((double)l[j] - (double)top) : 0.0;
                sum += s[j];
            }
            sum = wave_sum(sum);
#pragma unroll
            for (int j = 0; j < EPL; ++j) s[j] /= sum;
        } else {
#pragma unroll
            for (int j = 0; j < EPL; ++j) s[j] = 1.0 / (1.0 + exp(-(double)l[j]));
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = lane + 64 * j;
            const float b = a.bias && e < a.experts ? a.bias[e] : 0.0f;
            key[j] = l[j] > -INFINITY && b > -INFINITY ? ordered(s[j] + (double)b) : 0;
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) key[j] = l[j] > -INFINITY ? ordered(l[j]) : 0;
    }
    if (a.groups > 1) {
        Key worth = 0;   // lane g: group g's
        for (int g = 0; g < a.groups; ++g) {
            Key in[EPL], best = 0;
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                const int e = lane + 64 * j - g * a.group_size;
                in[j] = e >= 0 && e < a.group_size ? key[j] : 0;
                best = in[j] > best ? in[j] : best;
            }
            best = wave_umax(best);
            if constexpr (WIDE) {
                if (a.group_top2 && best != 0) {
                    const int at = first_with(in, best);
                    Key second = 0;
#pragma unroll
                    for (int j = 0; j < EPL; ++j) {
                        if (at == lane + 64 * j) in[j] = 0;
                        second = in[j] > second ? in[j] : second;
                    }
                    second = wave_umax(second);
                    if (second != 0) best = ordered(unordered(best) + unordered(second));
                }
            }
            if (lane == g) worth = best;
        }
        uint64_t kept = 0;
        for (int i = 0; i < a.topk_groups; ++i) {
            const Key w[1] = {worth};
            const Key best = wave_umax(worth);
            if (best == 0) break;
            const int g = first_with(w, best);
            kept |= 1ull << g;
            if (lane == g) worth = 0;
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            // e / group_size by its reciprocal: exact for e x group_size < 2^22
            const uint32_t g = ((uint32_t)(lane + 64 * j) * a.group_recip) >> 22;
            if (!(kept >> (g & 63) & 1)) key[j] = 0;
        }
    }
    my_id = -1;
    float my_l = -INFINITY;
    for (int i = 0; i < a.topk; ++i) {
        Key best = key[0];
#pragma unroll
        for (int j = 1; j < EPL; ++j) best = key[j] > best ? key[j] : best;
        best = wave_umax(best);
        if (best == 0) break;
        const int at = first_with(key, best);
        float li = 0.0f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            if (at == lane + 64 * j) key[j] = 0;
            if constexpr (WIDE) li = (at >> 6) == j ? l[j] : li;
        }
        if constexpr (WIDE) li = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(li), at & 63));
        else li = unordered(best);
        if (lane == i) {
            my_id = at;
            my_l = li;
        }
    }
    // weights: lane j holds the j-th choice
    const bool mine = my_id >= 0;
    float s;
    if (a.score == QLIN_SCORE_SOFTMAX) {
        // renormalized: the softmax over the chosen logits alone (the sum over
        // the others cancels), which does not underflow
        const float m = a.renormalize ? wave_max(my_l) : top;
        s = mine ? expf(my_l - m) : 0.0f;
        float sum = s;
        if (!a.renormalize) {
            sum = 0.0f;
#pragma unroll
            for (int j = 0; j < EPL; ++j) sum += l[j] > -INFINITY ? expf(l[j] - top) : 0.0f;
        }
        sum = wave_sum(sum);
        s = sum > 0.0f ? s / sum : 0.0f;
    } else {
        s = mine ? 1.0f / (1.0f + expf(-my_l)) : 0.0f;
        if (a.renormalize) {
            const float sum = wave_sum(s);
            s = sum > 0.0f ? s / sum : 0.0f;
        }
    }
    my_w = mine ? s * a.scale : 0.0f;
}

// Exclusive sums over value[0 .. n) (n <= kRouteThreads, one per thread) into
// off[0 .. n], by the whole workgroup.
__device__ __forceinline__ void scan_to(uint32_t value, int n, uint32_t *off, uint32_t *wave_tot) {
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    uint32_t v = tid < n ? value : 0;
    const uint32_t own = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t up = __shfl_up(v, d);
        if (lane >= d) v += up;
    }
    if (lane == 63) wave_tot[w] = v;
    __syncthreads();
    uint32_t before = 0;
    for (int i = 0; i < w; ++i) before += wave_tot[i];
    if (tid < n) off[tid] = before + v - own;
    if (tid == n - 1) off[n] = before + v;
    __syncthreads();
}

// Routes block_tokens tokens, 16 at a time (one per wave).  Each expert has a
// bit per token of the batch, so a pair's place among its expert's rows of
// this block is a count of bits: token order, whatever order waves come in.
//   one block:   scans the experts' counts and writes rows and slots
//   more blocks: leaves each pair's place in slots and the experts' counts
//                of this block in hist; place_kernel does the rest
template <int EPL, bool WIDE>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteLaunch a) {
    __shared__ uint32_t cnt[QLIN_MAX_EXPERTS], bits[QLIN_MAX_EXPERTS], off[QLIN_MAX_EXPERTS + 1];
    __shared__ uint32_t wave_tot[kRouteWaves];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    if (tid < a.experts) cnt[tid] = bits[tid] = 0;
    __syncthreads();
    const int t0 = blockIdx.x * a.block_tokens;
    const int t1 = min(a.T, t0 + a.block_tokens);
    for (int tb = t0; tb < t1; tb += kRouteWaves) {
        const int t = tb + w;
        int id = -1;
        float wt = 0.0f;
        if (t < t1) {
            route_token<EPL, WIDE>(a, t, lane, id, wt);
            if (lane < a.topk) {
                a.ids[(int64_t)t * a.topk + lane] = id;
                a.weights[(int64_t)t * a.topk + lane] = wt;
                if (id >= 0) atomicOr(&bits[id], 1u << w);
            }
        }
        __syncthreads();
        if (t < t1 && lane < a.topk)
            a.slots[(int64_t)t * a.topk + lane] =
                id >= 0 ? (int)(cnt[id] + __popc(bits[id] & ((1u << w) - 1))) : -1;
        __syncthreads();
        if (tid < a.experts) {
            cnt[tid] += __popc(bits[tid]);
            bits[tid] = 0;
        }
        __syncthreads();
    }
    if (gridDim.x > 1) {
        if (tid < a.experts) a.hist[(int64_t)blockIdx.x * a.experts + tid] = (uint16_t)cnt[tid];
        return;
    }
    scan_to(tid < a.experts ? cnt[tid] : 0, a.experts, off, wave_tot);
    for (int i = tid; i <= a.experts; i += kRouteThreads) a.offsets[i] = (int)off[i];
    for (int t = w; t < a.T; t += kRouteWaves) {
        if (lane >= a.topk) continue;
        const int64_t p = (int64_t)t * a.topk + lane;   // written by this thread above
        const int id = a.ids[p];
        if (id < 0) continue;
        const int slot = (int)off[id] + a.slots[p];
        a.slots[p] = slot;
        a.rows[slot] = t;
    }
    for (int i = (int)off[a.experts] + tid; i < a.T * a.topk; i += kRouteThreads) a.rows[i] = -1;
}

// Rows and slots of one block's pairs: the expert's offset, its rows in
// earlier blocks and the pair's place in its own block.  Every block sums the
// blocks' counts for itself (two bytes for each expert and block, out of the
// L2) instead of waiting for a third launch.
__global__ __launch_bounds__(kRouteThreads) void place_kernel(RouteLaunch a) {
    __shared__ uint32_t pre[QLIN_MAX_EXPERTS], tot[QLIN_MAX_EXPERTS], off[QLIN_MAX_EXPERTS + 1];
    __shared__ uint32_t wave_tot[kRouteWaves];
    const int tid = threadIdx.x;
    if (tid < a.experts) pre[tid] = tot[tid] = 0;
    __syncthreads();
    int width = 64;
    while (width < a.experts) width *= 2;
    const int e = tid & (width - 1), segs = kRouteThreads / width;
    if (e < a.experts) {
        uint32_t p = 0, s = 0;
        for (int b = tid / width; b < (int)gridDim.x; b += segs) {
            const uint32_t c = a.hist[(int64_t)b * a.experts + e];
            s += c;
            p += b < (int)blockIdx.x ? c : 0;
        }
        atomicAdd(&pre[e], p);
        atomicAdd(&tot[e], s);
    }
    __syncthreads();
    scan_to(tid < a.experts ? tot[tid] : 0, a.experts, off, wave_tot);
    if (blockIdx.x == 0)
        for (int i = tid; i <= a.experts; i += kRouteThreads) a.offsets[i] = (int)off[i];
    const int t0 = blockIdx.x * a.block_tokens;
    const int pairs = (min(a.T, t0 + a.block_tokens) - t0) * a.topk;
    for (int i = tid; i < pairs; i += kRouteThreads) {
        const int64_t p = (int64_t)t0 * a.topk + i;
        const int id = a.ids[p];
        if (id < 0) continue;
        const int slot = (int)(off[id] + pre[id]) + a.slots[p];
        a.slots[p] = slot;
        a.rows[slot] = t0 + i / a.topk;
    }
    for (int i = (int)off[a.experts] + (int)blockIdx.x * kRouteThreads + tid; i < a.T * a.topk;
         i += (int)gridDim.x * kRouteThreads)
        a.rows[i] = -1;
}

// ------------------------------------------------------------------ dispatch

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
                *reinterpret_cast<uint2 *>(a.xq + (int64_t)slot * a.K + c * 8) = q;
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
        *reinterpret_cast<uint2 *>(a.xq + (int64_t)slot * a.K + g * kGroup + j * 8) = q;
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

// eight elements at p as fp32, and back
template <bool F32>
__device__ __forceinline__ void load8(const void *base, int64_t at, float (&f)[8]) {
    if constexpr (F32) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + at);
        const float4 u = p[0], v = p[1];
        f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
        f[4] = v.x; f[5] = v.y; f[6] = v.z; f[7] = v.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + at);
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
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + at);
        p[0] = make_float4(f[0], f[1], f[2], f[3]);
        p[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + at) =
            make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
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

// Tokens per routing workgroup: all of them up to 64 (one launch, four
// batches of 16), else 16, or more so that there are at most 512 blocks to
// sum over.
int route_block_tokens(int T) {
    if (T <= 64) return 64;
    return 16 * ((T + 16 * 512 - 1) / (16 * 512));
}
int route_blocks(int T) { return T <= 64 ? 1 : (T + route_block_tokens(T) - 1) / route_block_tokens(T); }

hipError_t launch_route(const RouteLaunch &a, hipStream_t s) {
    const dim3 grid(route_blocks(a.T)), block(kRouteThreads);
    const bool wide = a.bias != nullptr || a.group_top2;
#define QLIN_ROUTE(EPL_)                                                                              \
    if (wide) hipLaunchKernelGGL((route_kernel<EPL_, true>), grid, block, 0, s, a);                   \
    else hipLaunchKernelGGL((route_kernel<EPL_, false>), grid, block, 0, s, a)
    if (a.experts <= 64) { QLIN_ROUTE(1); }
    else if (a.experts <= 128) { QLIN_ROUTE(2); }
    else if (a.experts <= 256) { QLIN_ROUTE(4); }
    else if (a.experts <= 512) { QLIN_ROUTE(8); }
    else { QLIN_ROUTE(16); }
#undef QLIN_ROUTE
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || grid.x == 1) return e;
    hipLaunchKernelGGL(place_kernel, grid, block, 0, s, a);
    return hipGetLastError();
}

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
        const int64_t groups = (int64_t)a.T * (a.K / kGroup);
        hipLaunchKernelGGL(dispatch_group_kernel, dim3((unsigned)((groups + 15) / 16)), dim3(256), 0, s, a);
    } else if (fmt == FMT_I8) {
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
