// qlin_rope.hip -- norms of the query and key heads with their rotation.
//
//   x' = x / sqrt(mean(x^2) + eps) * w,  (a, b) -> (a cos - b sin, b cos + a sin)
//
// Each element is read and written once and takes some ten operations, so the
// memory bounds it.  A head has 8, 16 or 32 lanes of 8 channels each, chosen so
// that both members of a rotated pair are one lane's: the only exchange is the
// sum of the squares.  From 1024 tokens on a workgroup has all heads of its token, so
// the angles are read once, and writes with the non-temporal policy: 8192 tokens of
// 72 heads of 128, bf16, 71.7 -> 62.3 -> 59.4 us (5.2 TB/s); with that policy on the
// reads instead 61.7.
#include "qlin_device.h"

namespace qlin {

namespace {

// A lane's two groups of four channels.  Rotated halves: 4 c and R / 2 + 4 c;
// rotated neighbours, and channels past R: 8 c and 8 c + 4.
template <bool F32>
__device__ __forceinline__ v4f load4(const void *base, int64_t at) {
    if constexpr (F32) return *reinterpret_cast<const v4f *>(static_cast<const float *>(base) + at);
    const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(base) + at);
    return v4f{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
}

typedef __bf16 v4bf __attribute__((ext_vector_type(4)));

template <bool F32, bool STREAM>
__device__ __forceinline__ void store4(void *base, int64_t at, v4f x) {
    if constexpr (F32) {
        v4f *to = reinterpret_cast<v4f *>(static_cast<float *>(base) + at);
        if constexpr (STREAM) __builtin_nontemporal_store(x, to);
        else *to = x;
    } else {
        const v4bf b = {(__bf16)x[0], (__bf16)x[1], (__bf16)x[2], (__bf16)x[3]};   // nearest even
        v4bf *to = reinterpret_cast<v4bf *>(static_cast<uint16_t *>(base) + at);
        if constexpr (STREAM) __builtin_nontemporal_store(b, to);
        else *to = b;
    }
}

// the sum over each aligned group of LANES lanes, in every one of them
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int d = 1; d < LANES; d *= 2) v += __shfl_xor(v, d);
    return v;
}

template <int LANES, bool IN32, bool OUT32, bool STREAM>
__global__ __launch_bounds__(256) void rope_kernel(RopeLaunch a) {
    constexpr int HEADS = 256 / LANES;      // heads of a step
    const int t = blockIdx.x;
    const int c = threadIdx.x % LANES, D = a.head_dim, R = a.rotary_dim;
    const int heads = a.q_heads + a.kv_heads;
    const int pos = R > 0 ? a.position[t] : 0;
    if (R > 0 && (unsigned)pos >= (unsigned)a.positions) return;   // padding
    const bool live = 8 * c < D, turned = 8 * c < R;
    const bool halves = turned && !a.interleaved;
    const int at0 = halves ? 4 * c : 8 * c, at1 = halves ? R / 2 + 4 * c : 8 * c + 4;
    v4f cs = {1, 1, 1, 1}, sn = {0, 0, 0, 0};
    if (turned) {
        const float *row = a.cos_sin + (int64_t)pos * R + 4 * c;
        cs = *reinterpret_cast<const v4f *>(row);
        sn = *reinterpret_cast<const v4f *>(row + R / 2);
    }
    for (int step = 0; step < a.steps; ++step) {
        const int h = (blockIdx.y * a.steps + step) * HEADS + threadIdx.x / LANES;
        const bool is_k = h >= a.q_heads, on = live && h < heads;
        const int64_t col = (int64_t)(is_k ? h - a.q_heads : h) * D;
        const int64_t from = (int64_t)t * (is_k ? a.ldk : a.ldq) + col;
        const int64_t to = (int64_t)t * (is_k ? a.ldko : a.ldqo) + col;
        const void *src = is_k ? a.k : a.q;
        const float *weight = is_k ? a.k_norm : a.q_norm;
        v4f x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
        if (on) {
            x = load4<IN32>(src, from + at0);
            y = load4<IN32>(src, from + at1);
        }
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += x[i] * x[i] + y[i] * y[i];
        sum = lanes_sum<LANES>(sum);
        if (weight && on) {
            const float norm = 1.0f / __builtin_sqrtf(sum / (float)D + a.eps);
            const v4f w0 = *reinterpret_cast<const v4f *>(weight + at0), w1 = *reinterpret_cast<const v4f *>(weight + at1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = x[i] * norm * w0[i];
                y[i] = y[i] * norm * w1[i];
            }
        }
        if (halves) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float u = x[i], v = y[i];
                x[i] = u * cs[i] - v * sn[i];
                y[i] = v * cs[i] + u * sn[i];
            }
        } else if (turned) {
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                float u = x[i], v = x[i + 1];
                x[i] = u * cs[i / 2] - v * sn[i / 2];
                x[i + 1] = v * cs[i / 2] + u * sn[i / 2];
                u = y[i], v = y[i + 1];
                y[i] = u * cs[2 + i / 2] - v * sn[2 + i / 2];
                y[i + 1] = v * cs[2 + i / 2] + u * sn[2 + i / 2];
            }
        }
        if (on) {
            void *dst = is_k ? a.k_out : a.q_out;
            store4<OUT32, STREAM>(dst, to + at0, x);
            store4<OUT32, STREAM>(dst, to + at1, y);
        }
    }
}

constexpr int kStreamTokens = 1024;

template <int LANES, bool STREAM>
void launch_types(bool in32, bool out32, const RopeLaunch &a, dim3 grid, hipStream_t s) {
    const dim3 block(256);
    if (in32 && out32) hipLaunchKernelGGL((rope_kernel<LANES, true, true, STREAM>), grid, block, 0, s, a);
    else if (in32) hipLaunchKernelGGL((rope_kernel<LANES, true, false, STREAM>), grid, block, 0, s, a);
    else if (out32) hipLaunchKernelGGL((rope_kernel<LANES, false, true, STREAM>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((rope_kernel<LANES, false, false, STREAM>), grid, block, 0, s, a);
}

template <int LANES>
void launch_lanes(bool in32, bool out32, RopeLaunch a, hipStream_t s) {
    constexpr int HEADS = 256 / LANES;
    const int groups = (a.q_heads + a.kv_heads + HEADS - 1) / HEADS;
    if (a.T >= kStreamTokens) {
        a.steps = groups;
        launch_types<LANES, true>(in32, out32, a, dim3(a.T, 1), s);
    } else {
        a.steps = 1;
        launch_types<LANES, false>(in32, out32, a, dim3(a.T, groups), s);
    }
}

}  // namespace

hipError_t launch_rope(bool in32, bool out32, const RopeLaunch &a, hipStream_t s) {
    if (a.head_dim <= 64) launch_lanes<8>(in32, out32, a, s);
    else if (a.head_dim <= 128) launch_lanes<16>(in32, out32, a, s);
    else launch_lanes<32>(in32, out32, a, s);
    return hipGetLastError();
}

}  // namespace qlin
