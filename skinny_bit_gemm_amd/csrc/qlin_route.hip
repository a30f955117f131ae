// qlin_route.hip -- routing tokens to experts: scores, top-k choice, weights,
// rows grouped by expert.
//
// The pages name MoE layers as the next target ("Building a High-Performance
// and Portable vLLM Linear Backend with Helion", section "Future work",
// model-coverage paragraph).
//
// Compiled with -fno-honor-nans: a maximum of doubles is then one instruction
// instead of two or three (8192 tokens, 256 experts in 8 groups: 20.4 us
// against 22.1).  No NaN takes part: the caller's logits and biases are loaded
// as integers, and a NaN among them has become -inf before it is a float
// (number_or_closed); what an all-closed token leaves in sums is not selected.
#include <algorithm>
#include <type_traits>

#include "qlin_device.h"

namespace qlin {

namespace {

constexpr int kPlaceThreads = 1024;
constexpr float kFltMax = 3.402823466e38f;
constexpr float kSigmoidZero = -709.782715f;   // e^709.782715 is past the largest double

// ---------------------------------------------- reductions over a token's lanes
//
// A token has LPT lanes: a wave (64) or a row of 16.  Every lane of the token
// gets the result.

// one DPP step of a maximum, a minimum or a sum (see max_dpp)
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ uint32_t moved_dpp(uint32_t v) {
    if constexpr (ROW_MASK == 0xF)   // every lane has a partner: nothing of the old value is needed
        return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
    else return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, ROW_MASK, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ float moved_dpp(float v) { return __uint_as_float(moved_dpp<CTRL, 0xF>(__float_as_uint(v))); }
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ uint32_t umax_dpp(uint32_t v) { return max(v, moved_dpp<CTRL, ROW_MASK>(v)); }
template <int CTRL>
__device__ __forceinline__ uint32_t umin_dpp(uint32_t v) { return min(v, moved_dpp<CTRL>(v)); }
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

template <int LPT>
__device__ __forceinline__ uint32_t token_max(uint32_t v) {
    v = umax_dpp<0xB1>(v);
    v = umax_dpp<0x4E>(v);
    v = umax_dpp<0x141>(v);
    v = umax_dpp<0x140>(v);
    if constexpr (LPT == 64) {
        v = umax_dpp<0x142, 0xA>(v);
        v = umax_dpp<0x143, 0xC>(v);
        v = (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
    }
    return v;
}
template <int LPT>
__device__ __forceinline__ uint64_t token_max(uint64_t v) {
    const uint32_t hi = token_max<LPT>((uint32_t)(v >> 32));
    const uint32_t lo = token_max<LPT>((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ uint32_t row16_min(uint32_t v) {
    v = umin_dpp<0xB1>(v);
    v = umin_dpp<0x4E>(v);
    v = umin_dpp<0x141>(v);
    return umin_dpp<0x140>(v);
}
template <int LPT>
__device__ __forceinline__ float token_max(float v) {
    if constexpr (LPT == 64) return wave_max(v);
    else return row16_max(v);
}
template <typename F>
__device__ __forceinline__ F row16_sum(F v) {
    v = add_dpp<0xB1>(v);
    v = add_dpp<0x4E>(v);
    v = add_dpp<0x141>(v);
    return add_dpp<0x140>(v);
}
template <int LPT>
__device__ __forceinline__ float token_sum(float v) {
    v = row16_sum(v);
    if constexpr (LPT == 64) {
        v = add_dpp<0x143, 0xC>(add_dpp<0x142, 0xA>(v));
        v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
    }
    return v;
}
template <int LPT>
__device__ __forceinline__ double token_sum(double v) {
    v = row16_sum(v);
    if constexpr (LPT == 64) {
        v = add_dpp<0x143, 0xC>(add_dpp<0x142, 0xA>(v));
        v = __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), 63),
                             __builtin_amdgcn_readlane(__double2loint(v), 63));
    }
    return v;
}

// 1 / d for d >= 1: two Newton steps from the hardware's estimate (within
// 2^-20 of itself or better, so within 2^-52 after them); 0 for infinity
__device__ __forceinline__ double recip(double d) {
    double y = __builtin_amdgcn_rcp(d);
    y = __builtin_fma(y, __builtin_fma(-d, y, 1.0), y);
    y = __builtin_fma(y, __builtin_fma(-d, y, 1.0), y);
    return d < INFINITY ? y : 0.0;
}

// p + q of what are products or exponentials, never fused into them: the two
// ways of routing a token have to get the same bits.
__device__ __forceinline__ double plus(double p, double q) {
#pragma clang fp contract(off)
    return p + q;
}

// The float of these bits, -inf where they are NaN's.
__device__ __forceinline__ float number_or_closed(uint32_t bits) {
    return __uint_as_float((bits & 0x7FFFFFFFu) > 0x7F800000u ? 0xFF800000u : bits);
}
__device__ __forceinline__ float bias_of(const RouteLaunch &a, int e) {
    return number_or_closed(reinterpret_cast<const uint32_t *>(a.bias)[e]);
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

// Lowest expert whose key is `best` (expert e = lane + 64 j): ballots in the
// order of j, then the lowest lane.
template <int EPL, typename Key>
__device__ __forceinline__ uint32_t first_with(const Key (&key)[EPL], Key best) {
    uint32_t at = 0;
#pragma unroll
    for (int j = EPL - 1; j >= 0; --j) {
        const uint64_t b = __ballot(key[j] == best);
        if (b) at = 64 * j + __ffsll((unsigned long long)b) - 1;
    }
    return at;
}

// The weight of the token's choice that this lane holds (my_id, logit my_l).
template <int LPT, int EPL>
__device__ __forceinline__ float weight_of(const RouteLaunch &a, const float (&l)[EPL], float top, int my_id, float my_l) {
    const bool mine = my_id >= 0;
    float s;
    if (a.score == QLIN_SCORE_SOFTMAX) {
        // renormalized: the softmax over the chosen logits alone (the sum over
        // the others cancels), which does not underflow
        const float m = a.renormalize ? token_max<LPT>(my_l) : top;
        s = mine ? expf(my_l - m) : 0.0f;
        float sum = s;
        if (!a.renormalize) {
            sum = 0.0f;
#pragma unroll
            for (int j = 0; j < EPL; ++j) sum += l[j] > -INFINITY ? expf(l[j] - top) : 0.0f;
        }
        sum = token_sum<LPT>(sum);
        s = sum > 0.0f ? s / sum : 0.0f;
    } else {
        // renormalized: times e^-m (m: the largest chosen logit, if negative),
        // which cancels and keeps what 32 bits would lose below -88.  What is 0
        // in 64 bits, where 1 + e^-l overflows, is 0 here.
        const float m = a.renormalize ? fminf(token_max<LPT>(my_l), 0.0f) : 0.0f;
        const float e = expf(-fabsf(my_l));
        s = mine && my_l > kSigmoidZero ? (my_l < 0.0f ? expf(my_l - m) : 1.0f) / (1.0f + e) : 0.0f;
        if (a.renormalize) {
            const float sum = token_sum<LPT>(s);
            s = sum > 0.0f ? s / sum : 0.0f;
        }
    }
    return mine ? s * a.scale : 0.0f;
}

// A token's logits: lane l holds experts l, l + LPT, ...; -inf where closed.
// Tokens past the call's (`live` false) are closed throughout.  Every lane
// loads, lanes without an expert the last one, so that no load has a branch.
template <int LPT, int EPL>
__device__ __forceinline__ void load_logits(const RouteLaunch &a, int t, bool live, int lane, float (&l)[EPL]) {
    const int64_t row = (int64_t)(live ? t : a.T - 1) * a.ld;
    uint32_t bits[EPL];
    if (a.logits_bf16) {
        const uint16_t *p = static_cast<const uint16_t *>(a.logits) + row;
#pragma unroll
        for (int j = 0; j < EPL; ++j) bits[j] = (uint32_t)p[min(lane + LPT * j, a.experts - 1)] << 16;
    } else {
        const uint32_t *p = static_cast<const uint32_t *>(a.logits) + row;
#pragma unroll
        for (int j = 0; j < EPL; ++j) bits[j] = p[min(lane + LPT * j, a.experts - 1)];
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j)
        l[j] = live && lane + LPT * j < a.experts ? fminf(number_or_closed(bits[j]), kFltMax) : -INFINITY;
}

// One token by a wave: lane j < topk ends with the j-th chosen expert
// (-1: none) and its weight.  Lane l holds experts l, l + 64, ...
template <int EPL, bool WIDE>
__device__ __forceinline__ void route_token(const RouteLaunch &a, int t, int lane, int &my_id, float &my_w) {
    using Key = std::conditional_t<WIDE, uint64_t, uint32_t>;
    float l[EPL];
    load_logits<64>(a, t, true, lane, l);
    float top = -INFINITY;
    if (a.score == QLIN_SCORE_SOFTMAX) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) top = fmaxf(top, l[j]);
        top = token_max<64>(top);
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
                sum = plus(sum, s[j]);
            }
            const double y = 1.0 / token_sum<64>(sum);
#pragma unroll
            for (int j = 0; j < EPL; ++j) s[j] *= y;
        } else {
#pragma unroll
            for (int j = 0; j < EPL; ++j) s[j] = recip(plus(1.0, exp(-(double)l[j])));
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = lane + 64 * j;
            const float b = a.bias && e < a.experts ? bias_of(a, e) : 0.0f;
            key[j] = l[j] > -INFINITY && b > -INFINITY ? ordered(plus(s[j], b)) : 0;
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) key[j] = l[j] > -INFINITY ? ordered(l[j]) : 0;
    }
    if (a.groups > 1) {
        uint64_t kept = 0;
        Key worth = 0;   // lane g: group g's
        for (int g = 0; g < a.groups; ++g) {
            Key in[EPL], best = 0;
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                const int e = lane + 64 * j - g * a.group_size;
                in[j] = e >= 0 && e < a.group_size ? key[j] : 0;
                best = in[j] > best ? in[j] : best;
            }
            best = token_max<64>(best);
            if constexpr (WIDE) {
                if (a.group_top2) {
                    const uint32_t at = first_with(in, best);
                    Key second = 0;
#pragma unroll
                    for (int j = 0; j < EPL; ++j) {
                        if (at == (uint32_t)(lane + 64 * j)) in[j] = 0;
                        second = in[j] > second ? in[j] : second;
                    }
                    second = token_max<64>(second);
                    if (best != 0 && second != 0) best = ordered(unordered(best) + unordered(second));
                }
            }
            if (g == lane) worth = best;
        }
        for (int n = 0; n < a.topk_groups; ++n) {
            const Key best = token_max<64>(worth);
            const uint32_t g = (uint32_t)__ffsll((unsigned long long)__ballot(worth == best)) - 1;
            if (best != 0) kept |= 1ull << (g & 63);
            if (g == (uint32_t)lane) worth = 0;
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
        best = token_max<64>(best);
        if (best == 0) break;
        const uint32_t at = first_with(key, best);
        float li = -INFINITY;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const bool here = at == (uint32_t)(lane + 64 * j);
            if constexpr (WIDE) li = here ? l[j] : li;
            if (here) key[j] = 0;
        }
        if constexpr (WIDE) li = token_max<64>(li);
        else li = unordered(best);
        if (lane == i) {
            my_id = (int)at;
            my_l = li;
        }
    }
    my_w = weight_of<64, EPL>(a, l, top, my_id, my_l);
}

// One DPP step's partner of a double.
template <int CTRL>
__device__ __forceinline__ double moved_dpp(double v) {
    return __hiloint2double((int)moved_dpp<CTRL, 0xF>((uint32_t)__double2hiint(v)),
                            (int)moved_dpp<CTRL, 0xF>((uint32_t)__double2loint(v)));
}
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return fmin(a, b); }
template <typename C>
__device__ __forceinline__ C row_max(C v) {
    v = larger(v, moved_dpp<0xB1>(v));
    v = larger(v, moved_dpp<0x4E>(v));
    v = larger(v, moved_dpp<0x141>(v));
    return larger(v, moved_dpp<0x140>(v));
}

// What a score becomes once its expert is taken: the lowest float, or a double
// below -2^1023 whose low word stays as it was.
__device__ __forceinline__ float taken(bool now, float c) { return now ? -INFINITY : c; }
__device__ __forceinline__ double taken(bool now, double c) {
    return __hiloint2double(now ? (int)0xFFEFFFFF : __double2hiint(c), __double2loint(c));
}

// One token by a row of 16 lanes, where four tokens share each instruction of
// the reductions (groups of a multiple of 16 experts, at most 16 of them).  The
// scores are compared as numbers, in 64 bits (WIDE) where their sums need it:
// a double's maximum is one instruction.  They have the bits that route_token
// gives them, a softmax's sum in the same order (sum[q]: the experts that a
// wave has in its row q), so a token chooses the same in a call of any size.
template <int EPL, bool WIDE>
__device__ __forceinline__ void route_row(const RouteLaunch &a, int t, bool live, int lane, int &my_id, float &my_w) {
    using C = std::conditional_t<WIDE, double, float>;
    constexpr C kClosed = -INFINITY;
    constexpr C kTaken = WIDE ? (C)-0x1p1023 : (C)-INFINITY;   // no score is this low
    float l[EPL];
    C c[EPL];
    load_logits<16>(a, t, live, lane, l);
    float top = -INFINITY;
    if (a.score == QLIN_SCORE_SOFTMAX) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) top = fmaxf(top, l[j]);
        top = row16_max(top);
    }
    if constexpr (WIDE) {
        if (a.score == QLIN_SCORE_SOFTMAX) {
            double sum[4] = {};
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                c[j] = l[j] > -INFINITY ? exp((double)l[j] - (double)top) : 0.0;
                sum[j & 3] = plus(sum[j & 3], c[j]);
            }
            const double y = 1.0 / ((row16_sum(sum[3]) + row16_sum(sum[2])) + (row16_sum(sum[1]) + row16_sum(sum[0])));
#pragma unroll
            for (int j = 0; j < EPL; ++j) c[j] *= y;
        } else {
#pragma unroll
            for (int j = 0; j < EPL; ++j) c[j] = recip(plus(1.0, exp(-(double)l[j])));
        }
        if (a.bias) {
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                const float b = bias_of(a, min(lane + 16 * j, a.experts - 1));
                c[j] = b > -INFINITY ? plus(c[j], b) : kClosed;
            }
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j) c[j] = l[j] > -INFINITY ? c[j] : kClosed;
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) c[j] = l[j];
    }
    if (a.groups > 1) {
        const int per = a.group_size >> 4;   // numbers j of a group
        C worth = kClosed, m1 = kClosed, m2 = kClosed;   // worth: lane g, group g's
        int g = 0, left = per;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            m2 = larger(m2, smaller(m1, c[j]));
            m1 = larger(m1, c[j]);
            if (--left == 0) {   // the two largest of the group, over the row
                auto merge = [&](C o1, C o2) {
                    m2 = larger(smaller(m1, o1), larger(m2, o2));
                    m1 = larger(m1, o1);
                };
                merge(moved_dpp<0xB1>(m1), moved_dpp<0xB1>(m2));
                merge(moved_dpp<0x4E>(m1), moved_dpp<0x4E>(m2));
                merge(moved_dpp<0x141>(m1), moved_dpp<0x141>(m2));
                merge(moved_dpp<0x140>(m1), moved_dpp<0x140>(m2));
                const C both = a.group_top2 && m2 > kClosed ? m1 + m2 : m1;
                worth = lane == g ? both : worth;
                m1 = m2 = kClosed;
                ++g;
                left = per;
            }
        }
        uint32_t kept = 0;
        for (int n = 0; n < a.topk_groups; ++n) {
            const C best = row_max(worth);
            const uint32_t at = row16_min(worth == best ? (uint32_t)lane : 99u);
            if (best > kClosed) kept |= 1u << at;
            if ((uint32_t)lane == at) worth = kClosed;
        }
        g = 0;
        left = per;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            if (!(kept >> g & 1)) c[j] = kClosed;
            if (--left == 0) {
                ++g;
                left = per;
            }
        }
    }
    my_id = -1;
    for (int i = 0; i < a.topk; ++i) {
        C best = c[0];
#pragma unroll
        for (int j = 1; j < EPL; ++j) best = larger(best, c[j]);
        best = row_max(best);
        // the lowest expert with it: this lane's first, then the lowest of the
        // row; the comparisons' lane masks say which number is taken
        bool here[EPL];
        uint32_t mine = 0xFFFF;
#pragma unroll
        for (int j = EPL - 1; j >= 0; --j) {
            here[j] = c[j] == best;
            mine = here[j] ? lane + 16 * j : mine;
        }
        const uint32_t at = row16_min(mine);
        bool owner = at == mine;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            c[j] = taken(owner && here[j], c[j]);
            owner = owner && !here[j];
        }
        if (lane == i && best > kTaken) my_id = (int)at;
    }
    float my_l = -INFINITY;
    if (my_id >= 0) {
        const int64_t at = (int64_t)t * a.ld + my_id;
        my_l = a.logits_bf16 ? __uint_as_float((uint32_t) static_cast<const uint16_t *>(a.logits)[at] << 16)
                             : static_cast<const float *>(a.logits)[at];
        my_l = fminf(my_l, kFltMax);
    }
    my_w = weight_of<16, EPL>(a, l, top, my_id, my_l);
}

// Exclusive sums over value (one per thread, n <= the workgroup's threads)
// into off[0 .. n].
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

template <int LPT, int EPL, bool WIDE>
__device__ __forceinline__ void route_any(const RouteLaunch &a, int t, bool live, int lane, int &id, float &w) {
    if constexpr (LPT == 16) {
        if (__any(live)) route_row<EPL, WIDE>(a, t, live, lane, id, w);
    } else {
        if (live) route_token<EPL, WIDE>(a, t, lane, id, w);
    }
}

// Routes block_tokens tokens, TOKENS at a time.  Each expert has a bit per
// token of these, so a pair's place among its expert's rows of this block is a
// count of bits: token order, whatever order the waves come in.  Leaves each
// pair's place in slots and the experts' counts of this block in hist;
// place_kernel does the rest.
template <int LPT, int EPL, bool WIDE, int TOKENS>
__global__ __launch_bounds__(TOKENS *LPT) void route_kernel(RouteLaunch a) {
    static_assert(TOKENS <= 32, "a bit per token");
    constexpr int THREADS = TOKENS * LPT;
    __shared__ uint32_t cnt[QLIN_MAX_EXPERTS], bits[QLIN_MAX_EXPERTS];
    const int tid = threadIdx.x, lane = tid % LPT, w = tid / LPT;
    for (int e = tid; e < a.experts; e += THREADS) cnt[e] = bits[e] = 0;
    __syncthreads();
    const int t0 = blockIdx.x * a.block_tokens;
    const int t1 = min(a.T, t0 + a.block_tokens);
    for (int tb = t0; tb < t1; tb += TOKENS) {
        const int t = tb + w;
        const bool live = t < t1;
        int id = -1;
        float wt = 0.0f;
        route_any<LPT, EPL, WIDE>(a, t, live, lane, id, wt);
        if (live && lane < a.topk) {
            a.ids[(int64_t)t * a.topk + lane] = id;
            a.weights[(int64_t)t * a.topk + lane] = wt;
            if (id >= 0) atomicOr(&bits[id], 1u << w);
        }
        __syncthreads();
        if (live && lane < a.topk)
            a.slots[(int64_t)t * a.topk + lane] =
                id >= 0 ? (int)(cnt[id] + __popc(bits[id] & ((1u << w) - 1))) : -1;
        __syncthreads();
        for (int e = tid; e < a.experts; e += THREADS) {
            cnt[e] += __popc(bits[e]);
            bits[e] = 0;
        }
        __syncthreads();
    }
    for (int e = tid; e < a.hist_stride; e += THREADS)
        a.hist[(int64_t)blockIdx.x * a.hist_stride + e] = e < a.experts ? (uint16_t)cnt[e] : 0;
}

// All of the call's tokens (at most 64) at once, by one workgroup: one launch.
// As route_kernel, with the sums over the experts added.
template <int LPT, int EPL, bool WIDE>
__global__ __launch_bounds__(1024) void route_once_kernel(RouteLaunch a) {
    __shared__ uint32_t bits[2][QLIN_MAX_EXPERTS], off[QLIN_MAX_EXPERTS + 1], wave_tot[16];
    const int tid = threadIdx.x, lane = tid % LPT, t = tid / LPT, threads = blockDim.x;
    for (int e = tid; e < a.experts; e += threads) bits[0][e] = bits[1][e] = 0;
    const bool live = t < a.T;
    int id = -1;
    float wt = 0.0f;
    route_any<LPT, EPL, WIDE>(a, t, live, lane, id, wt);
    __syncthreads();
    if (live && lane < a.topk) {
        a.ids[t * a.topk + lane] = id;
        a.weights[t * a.topk + lane] = wt;
        if (id >= 0) atomicOr(&bits[t >> 5][id], 1u << (t & 31));
    }
    __syncthreads();
    scan_to(tid < a.experts ? __popc(bits[0][tid]) + __popc(bits[1][tid]) : 0, a.experts, off, wave_tot);
    if (live && lane < a.topk) {
        int slot = -1;
        if (id >= 0) {
            const uint32_t below = (1u << (t & 31)) - 1;
            slot = (int)(off[id] + (t < 32 ? __popc(bits[0][id] & below) : __popc(bits[0][id]) + __popc(bits[1][id] & below)));
            a.rows[slot] = t;
        }
        a.slots[t * a.topk + lane] = slot;
    }
    for (int i = tid; i <= a.experts; i += threads) a.offsets[i] = (int)off[i];
    for (int i = (int)off[a.experts] + tid; i < a.T * a.topk; i += threads) a.rows[i] = -1;
}

// Rows and slots of the pairs of kPlaceBlocks routing blocks: the expert's
// offset, its rows in earlier blocks and the pair's place in its own block.
// Every workgroup sums the blocks' counts for itself (2 bytes for each expert
// and block, out of the L2) instead of waiting for a third launch.
constexpr int kPlaceBlocks = 8;

__global__ __launch_bounds__(kPlaceThreads) void place_kernel(RouteLaunch a) {
    __shared__ uint32_t pre[QLIN_MAX_EXPERTS], tot[QLIN_MAX_EXPERTS], off[QLIN_MAX_EXPERTS + 1];
    __shared__ __align__(16) uint16_t own[kPlaceBlocks][QLIN_MAX_EXPERTS];   // counts, then places, of this workgroup's blocks
    __shared__ uint32_t wave_tot[16];
    const int tid = threadIdx.x;
    const int b0 = blockIdx.x * kPlaceBlocks, b1 = min(a.blocks, b0 + kPlaceBlocks);
    const int t0 = b0 * a.block_tokens;
    const int pairs = (min(a.T, b1 * a.block_tokens) - t0) * a.topk;
    // the first pairs are on their way while the counts are summed
    constexpr int kAhead = 2;
    int ahead_id[kAhead], ahead_place[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
        const int i = q * kPlaceThreads + tid;
        ahead_id[q] = i < pairs ? a.ids[(int64_t)t0 * a.topk + i] : -1;
        ahead_place[q] = i < pairs ? a.slots[(int64_t)t0 * a.topk + i] : 0;
    }
    if (tid < a.hist_stride) pre[tid] = tot[tid] = 0;
    __syncthreads();
    const int cols = a.hist_stride / 8, segs = kPlaceThreads / cols;
    const int col = tid % cols, seg = tid / cols;
    if (seg < segs) {
        uint32_t p[8] = {}, s[8] = {};
        for (int first = seg; first < a.blocks; first += 8 * segs) {
            uint4 v[8];   // eight loads on their way at a time
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int b = first + u * segs;
                v[u] = make_uint4(0, 0, 0, 0);
                if (b < a.blocks) v[u] = *reinterpret_cast<const uint4 *>(a.hist + (int64_t)b * a.hist_stride + col * 8);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int b = first + u * segs;
                const uint32_t q[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t c = i & 1 ? q[i / 2] >> 16 : q[i / 2] & 0xFFFFu;
                    s[i] += c;
                    p[i] += b < b0 ? c : 0;
                }
                if (b >= b0 && b < b1) *reinterpret_cast<uint4 *>(&own[b - b0][col * 8]) = v[u];
            }
        }
        // expert 8 col + i lies at i x cols + col: neighbouring lanes add in
        // neighbouring banks
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            atomicAdd(&pre[i * cols + col], p[i]);
            atomicAdd(&tot[i * cols + col], s[i]);
        }
    }
    __syncthreads();
    scan_to(tid < a.experts ? tot[(tid & 7) * cols + (tid >> 3)] : 0, a.experts, off, wave_tot);
    if (blockIdx.x == 0)
        for (int i = tid; i <= a.experts; i += kPlaceThreads) a.offsets[i] = (int)off[i];
    if (tid < a.experts) {
        uint32_t at = 0;
        for (int b = 0; b < b1 - b0; ++b) {
            const uint32_t c = own[b][tid];
            own[b][tid] = (uint16_t)at;
            at += c;
        }
    }
    __syncthreads();
    auto put = [&](int i, int id, int place) {
        if (id < 0) return;
        const int t = i / a.topk;
        const int slot = (int)(off[id] + pre[(id & 7) * cols + (id >> 3)] + own[t / a.block_tokens][id]) + place;
        a.slots[(int64_t)t0 * a.topk + i] = slot;
        a.rows[slot] = t0 + t;
    };
#pragma unroll
    for (int q = 0; q < kAhead; ++q) put(q * kPlaceThreads + tid, ahead_id[q], ahead_place[q]);
    for (int i = kAhead * kPlaceThreads + tid; i < pairs; i += kPlaceThreads)
        put(i, a.ids[(int64_t)t0 * a.topk + i], a.slots[(int64_t)t0 * a.topk + i]);
    for (int i = (int)off[a.experts] + (int)blockIdx.x * kPlaceThreads + tid; i < a.T * a.topk;
         i += (int)gridDim.x * kPlaceThreads)
        a.rows[i] = -1;
}

}  // namespace

// --------------------------------------------------------------- launchers

// How a call runs (times: inside a replayed graph).
//   rows   16 lanes per token (route_row) instead of a wave: past 8 tokens,
//          where four tokens share an instruction (256 experts with a bias,
//          16 tokens: 7.1 us against 9.6; 4 tokens: 7.0 against 6.4), and for
//          a wave that would have a single number in a lane or a group at a
//          time (256 in 8 groups, 1 token: 8.8 us against 10.8, 4096 tokens:
//          16.4 against 24.6; 60 experts, 64 tokens: 4.5 against 8.5)
//   once   one launch for all tokens by one workgroup: 64 of them with 16
//          lanes each (64 tokens, 60 experts with a bias: 6.2 us against 8.5
//          in two launches, 128: 8.4 against 8.8; 256: 7.0 against 8.4 without
//          a bias, but 12.9 against 10.8 with one), 32 with groups, whose
//          choice is longer (256 in 8, 64 tokens: 19.3 against 13.7), 16 with
//          a wave each
//   else   blocks of block_tokens tokens and a second launch: 16 tokens as
//          long as there is a compute unit for each block (256 in 8 groups,
//          1024 tokens: 15.8 us against 19.7 with 32), then 32 (8192: 20.5
//          against 21.8 with 16); at most 512 blocks to sum over
constexpr int kMostBlocks = 512;

RoutePlan route_plan(const qlin_router &r, int T) {
    RoutePlan p = {};
    const int group = r.experts / r.groups;
    const bool fits = r.experts <= 256 && r.topk <= 16 && (r.groups == 1 || (r.groups <= 16 && group % 16 == 0));
    p.rows = fits && (T > 8 || r.experts <= 64 || r.groups > 1);
    p.once = T <= (!p.rows ? 16 : r.groups > 1 ? 32 : 64);
    const int tokens = p.rows && T > 16 * kComputeUnits ? 32 : 16;
    p.block_tokens = tokens * ((T + tokens * kMostBlocks - 1) / (tokens * kMostBlocks));
    p.blocks = p.once ? 1 : (T + p.block_tokens - 1) / p.block_tokens;
    // no call of at most T tokens has more blocks than this: a workspace for
    // the most tokens serves fewer
    p.ws_blocks = p.once ? 0 : std::min((T + 15) / 16, kMostBlocks);
    return p;
}

template <int LPT, int EPL, int TOKENS>
static void launch_route_blocks(const RouteLaunch &a, bool wide, hipStream_t s) {
    const dim3 grid(a.blocks), block(TOKENS * LPT);
    if (wide) hipLaunchKernelGGL((route_kernel<LPT, EPL, true, TOKENS>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((route_kernel<LPT, EPL, false, TOKENS>), grid, block, 0, s, a);
}

template <int LPT, int EPL>
static void launch_route_kernel(const RouteLaunch &a, bool once, hipStream_t s) {
    const bool wide = a.bias != nullptr || a.group_top2;
    if (once) {
        // as many threads as the tokens and the sums over the experts need
        const int need = std::max(a.T * LPT, a.experts);
        const dim3 block((std::max(need, 64) + 63) / 64 * 64);
        if (wide) hipLaunchKernelGGL((route_once_kernel<LPT, EPL, true>), dim3(1), block, 0, s, a);
        else hipLaunchKernelGGL((route_once_kernel<LPT, EPL, false>), dim3(1), block, 0, s, a);
    } else {
        if (LPT == 16 && a.block_tokens > 16) launch_route_blocks<LPT, EPL, LPT == 16 ? 32 : 16>(a, wide, s);
        else launch_route_blocks<LPT, EPL, 16>(a, wide, s);
    }
}

hipError_t launch_route(const RoutePlan &p, const RouteLaunch &a, hipStream_t s) {
    if (p.rows) {
        if (a.experts <= 64) launch_route_kernel<16, 4>(a, p.once, s);
        else if (a.experts <= 128) launch_route_kernel<16, 8>(a, p.once, s);
        else launch_route_kernel<16, 16>(a, p.once, s);
    } else {
        if (a.experts <= 64) launch_route_kernel<64, 1>(a, p.once, s);
        else if (a.experts <= 128) launch_route_kernel<64, 2>(a, p.once, s);
        else if (a.experts <= 256) launch_route_kernel<64, 4>(a, p.once, s);
        else if (a.experts <= 512) launch_route_kernel<64, 8>(a, p.once, s);
        else launch_route_kernel<64, 16>(a, p.once, s);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.once) return e;
    hipLaunchKernelGGL(place_kernel, dim3((a.blocks + kPlaceBlocks - 1) / kPlaceBlocks), dim3(kPlaceThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace qlin
